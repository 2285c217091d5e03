"""Attention over the paged cache (include/q4k_layer.h) against 64 bits: prompts,
chunks, single tokens and trees of drafted tokens."""
import numpy as np
import pytest

import gguf_q4_dequant_amd as q4k
from tests.gpu_helpers import to_dev
from tests.layer_reference import TYPES, Paged, attention, rng_of, tolerance, tree_mask

pytestmark = pytest.mark.gpu


def run(p, q, scale, mask=None, out=None):
    cache, seqs = p.on_device()
    if mask is None:
        return q4k.attention(to_dev(q), cache, seqs, scale, out=out)
    return q4k.attention_tree(to_dev(q), cache, seqs, to_dev(mask.view(np.int32)), scale, out=out)


def check(p, rng, q_heads, mask=None, words=0, scale=None, big=1.0):
    import torch
    q = (big * rng.standard_normal((p.T, q_heads, p.D))).astype(np.float32)
    sentinel = torch.full(q.shape, 7.25, device="cuda")
    got = run(p, q, scale, mask, sentinel).cpu().numpy()
    n = min(max(int(p.offsets[-1]), 0), p.T)
    with np.errstate(invalid="ignore"):
        want, S, A = attention(p, q, p.D ** -0.5 if scale is None else scale, mask, words)
    assert (got[n:] == 7.25).all()
    got, want, S, A = got[:n], want[:n], S[:, :n], A[:n]
    off, tol = np.abs(got - want), tolerance(p, S, A, int(max(p.lengths.max(), 1)))
    lost = ~np.isfinite(want)  # a row that sees NaN or an infinity (places behind a sequence's end hold them)
    bad = np.where(lost, np.isfinite(got), ~(off <= tol))
    assert not bad.any(), (int(bad.sum()), bad.size, np.argwhere(bad)[:4].tolist(), got[bad][:4], want[bad][:4], tol[bad][:4])
    return got


SETS = {
    "one token": [(1000, 1)],
    "first token": [(0, 1)],
    "short contexts": [(b, 1) for b in range(20)],
    "batch": [(700, 1), (0, 1), (63, 1), (64, 1), (65, 1), (2500, 1), (31, 1)],
    "prompt": [(0, 200)],
    "prompts": [(0, 37), (0, 1), (0, 130), (0, 64)],
    "chunk": [(300, 32)],
    "ragged": [(5, 3), (0, 0), (64, 1), (131, 18), (0, 2), (600, 65), (0, 0)],
    "before the start": [(-3, 5), (-2, 2), (-1, 1), (-7, 40), (4, 2)],
}


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("group", [1, 4])
@pytest.mark.parametrize("name", SETS)
def test_causal(name, group, kind):
    rng = rng_of(20, list(SETS).index(name), group, TYPES.index(kind))
    scales = (0.05, 0.07) if kind == "e4m3" else (1.0, 1.0)
    check(Paged(rng, SETS[name], 2, 64, 16, kind, *scales, extra_rows=2, extra_cols=1), rng, 2 * group)


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("D", [16, 32, 48, 64, 80, 96, 112, 128, 160, 192, 240, 256])
def test_head_sizes(D, kind):
    rng = rng_of(21, D, TYPES.index(kind))
    check(Paged(rng, [(150, 1), (20, 3)], 2, D, 16, kind), rng, 6)
    check(Paged(rng, [(70, 90), (0, 33)], 1, D, 32, kind), rng, 2)


@pytest.mark.parametrize("group", [1, 2, 3, 5, 7, 8, 12, 16, 17, 40, 71])
def test_groups(group):
    rng = rng_of(22, group)
    check(Paged(rng, [(333, 1), (90, 2)], 1, 64, 16, "f16"), rng, group)
    check(Paged(rng, [(33, 50)], 1, 64, 16, "bf16"), rng, group)


@pytest.mark.parametrize("page", [1, 2, 8, 16, 128, 1024])
def test_page_sizes(page):
    rng = rng_of(23, page)
    check(Paged(rng, [(170, 1), (1, 1)], 2, 64, page, "f16"), rng, 4)
    check(Paged(rng, [(70, 79), (1, 70)], 2, 64, page, "bf16"), rng, 4)


@pytest.mark.parametrize("kind", TYPES)
def test_long_contexts(kind):
    rng = rng_of(24, TYPES.index(kind))
    check(Paged(rng, [(9000, 1)], 1, 128, 64, kind), rng, 5)
    check(Paged(rng, [(5000, 4), (17, 2), (2100, 1)], 2, 64, 16, kind), rng, 8)
    check(Paged(rng, [(4000, 40)], 1, 64, 64, kind), rng, 4)


def test_many_sequences():
    rng = rng_of(25)
    check(Paged(rng, [(int(rng.integers(0, 90)), int(rng.integers(0, 3))) for _ in range(200)], 1, 32, 8, "f16"), rng, 2)
    check(Paged(rng, [(int(rng.integers(0, 9)), int(rng.integers(0, 30))) for _ in range(130)], 1, 32, 8, "bf16"), rng, 2)


@pytest.mark.parametrize("kind", TYPES)
def test_scores_far_apart(kind):
    """Large queries: scores of hundreds, almost one weight a row; and a scale of its own, negative and zero."""
    rng = rng_of(26, TYPES.index(kind))
    p = Paged(rng, [(100, 1), (30, 40)], 2, 64, 16, kind)
    check(p, rng, 4, big=300.0)
    check(p, rng, 4, scale=-0.3)
    check(p, rng, 4, scale=0.0)
    check(p, rng, 4, scale=1e-8, big=1e6)


def test_tiny_and_huge_values():
    """Queries and scales far outside binary16's range: rows are scaled by powers of two."""
    rng = rng_of(27)
    p = Paged(rng, [(100, 1), (30, 40)], 2, 64, 16, "f16")
    for big, scale in ((1e-12, 1e11), (1e12, 1e-13), (1e-20, 1.0), (3e20, 1e-21)):
        check(p, rng, 4, scale=scale, big=big)


TREES = {
    "one": [(90, 8)],
    "no context": [(0, 9), (0, 1)],
    "wide": [(200, 40), (5, 33), (0, 64), (77, 1), (0, 0), (1000, 63)],
    "long": [(3000, 16)],
}


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("group", [1, 4])
@pytest.mark.parametrize("name", TREES)
def test_tree(name, group, kind):
    rng = rng_of(30, list(TREES).index(name), group, TYPES.index(kind))
    sizes = TREES[name]
    for words in (2, 3):
        mask = tree_mask(rng, sizes, words, 2)
        check(Paged(rng, sizes, 2, 64, 16, kind, extra_rows=2), rng, 2 * group, mask, words)


@pytest.mark.parametrize("D", [48, 128, 256])
def test_tree_head_sizes(D):
    rng = rng_of(31, D)
    sizes = [(100, 12), (3, 20)]
    check(Paged(rng, sizes, 2, D, 16, "bf16"), rng, 4, tree_mask(rng, sizes, 1), 1)


def test_masks_of_every_kind():
    """Random bits (later tokens seen, the token itself not), empty rows with and without
    a context, and new tokens behind the mask's words."""
    rng = rng_of(32)
    sizes = [(0, 50), (20, 50), (0, 3), (130, 70)]
    T = sum(n for _, n in sizes)
    mask = rng.integers(0, 1 << 32, (T, 2), dtype=np.uint32)
    mask[::5] = 0
    got = check(Paged(rng, sizes, 2, 64, 16, "f16"), rng, 4, mask, 2)
    assert (got[0] == 0).all()
    check(Paged(rng, sizes, 2, 64, 16, "f16"), rng, 4, mask[:, :1].copy(), 1)


def test_lower_triangle_as_a_tree_is_causal():
    import torch
    rng = rng_of(33)
    sizes = [(100, 40), (0, 25)]
    p = Paged(rng, sizes, 2, 64, 16, "f16")
    q = rng.standard_normal((65, 4, 64)).astype(np.float32)
    mask = np.array([[(2 << i) - 1 & 0xFFFFFFFF, (2 << i) - 1 >> 32] for _, n in sizes for i in range(n)], np.uint32)
    assert torch.allclose(run(p, q, None), run(p, q, None, mask), rtol=2e-5, atol=2e-5)


def test_missing_pages_are_masked():
    rng = rng_of(34)
    for sizes in ([(300, 1), (200, 1), (90, 1), (100, 1)], [(100, 40), (0, 70), (20, 30), (64, 64)]):
        p = Paged(rng, sizes, 2, 64, 16, "f16")
        p.table[0, 1] = -1
        p.table[0, 3] = p.pool
        p.table[1, :] = -1                        # nothing left: zeros
        p.table[2, 0] = 2 ** 31 - 1
        p.lengths[3] = 16 * p.table.shape[1] + 9  # longer than the table
        got = check(p, rng, 4)  # and then sees what is behind it in its last page
        first, end = p.offsets[1], p.offsets[2]
        assert (got[first:end] == 0).all()
        p.table = p.table[:, :0]
        assert (check(p, rng, 4)[:p.T] == 0).all()


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("what", ["k", "v"])
def test_what_is_not_seen_never_reaches_a_row(what, kind):
    """NaN and infinities in a later token's keys or values: the rows before it are
    what they are without, and the rows that see it show it."""
    import torch
    rng = rng_of(35, TYPES.index(kind))
    sizes = [(40, 50), (0, 90)]
    mask = tree_mask(rng, sizes, 3)
    for m in (None, mask):
        for value in (np.nan, np.inf, -np.inf):
            p = Paged(rng, sizes, 2, 64, 16, kind)
            q = rng.standard_normal((p.T, 8, 64)).astype(np.float32)
            clean = run(p, q, None, m).cpu().numpy()
            i = 20  # the new token of sequence 1 whose key or value is bad
            at = p.table[1, i // 16], i % 16
            t = getattr(p, what)
            t[at[0], 1, at[1], 5] = torch.tensor(value).to(t.dtype)
            got = run(p, q, None, m).cpu().numpy()
            see = np.zeros(p.T, bool)
            see[50 + i:] = True if m is None else (m[50 + i:, 0] >> i & 1) == 1
            assert np.array_equal(got[~see], clean[~see])
            assert np.array_equal(got[:, :4], clean[:, :4])  # the other key head
            isnan = kind == "e4m3" or np.isnan(value)
            if what == "v":
                assert not np.isfinite(got[see][:, 4:, 5]).any()
                keep = np.arange(64) != 5
                assert np.array_equal(got[see][:, :, keep], clean[see][:, :, keep])
            elif isnan:
                assert np.isnan(got[see][:, 4:]).all()


def test_nan_queries_stay_in_their_rows():
    rng = rng_of(36)
    p = Paged(rng, [(40, 3), (0, 30)], 2, 64, 16, "f16")
    q = rng.standard_normal((33, 4, 64)).astype(np.float32)
    clean = run(p, q, None).cpu().numpy()
    for value in (np.nan, np.inf):
        bad = q.copy()
        bad[1, 2, 7] = bad[20, 0, 0] = value
        got = run(p, bad, None).cpu().numpy()
        hit = np.zeros((33, 4), bool)
        hit[1, 2] = hit[20, 0] = True
        assert np.isnan(got[hit]).all() and np.array_equal(got[~hit], clean[~hit])


def test_the_same_call_gives_the_same_bits():
    import torch
    rng = rng_of(37)
    p = Paged(rng, [(3000, 1), (100, 1), (900, 1)], 2, 128, 32, "f16")
    q = rng.standard_normal((3, 16, 128)).astype(np.float32)
    first = run(p, q, None)
    assert all(torch.equal(run(p, q, None), first) for _ in range(5))


def test_shared_pages():
    """Two sequences with a common prefix in the same pages."""
    rng = rng_of(38)
    p = Paged(rng, [(64, 1), (64, 9), (64, 1)], 2, 64, 16, "f16")
    p.table[1, :4] = p.table[0, :4]
    p.table[2, :4] = p.table[0, :4]
    check(p, rng, 8)


def test_offsets_past_32_bits():
    """Pages at the end of a pool of more than 2^32 elements."""
    import torch
    page, heads, D = 1024, 2, 128
    pages = (1 << 32) // (page * heads * D) + 3
    pool = torch.full((pages, heads, page, D), float("nan"), dtype=torch.float8_e4m3fn, device="cuda")
    rng = rng_of(39)
    for sizes in ([(1200, 1)], [(900, 300)]):
        small = Paged(rng, sizes, heads, D, page, "e4m3", spare=0)
        q = to_dev(rng.standard_normal((small.T, 4, D)).astype(np.float32))
        cache, seqs = small.on_device()
        want = q4k.attention(q, cache, seqs)
        pool[pages - 2:] = cache.k[:2]
        big_v = pool.clone()
        big_v[pages - 2:] = cache.v[:2]
        far = q4k.Sequences(seqs.offsets, seqs.lengths, seqs.pages + (pages - 2))
        assert torch.equal(q4k.attention(q, q4k.KVCache(pool, big_v), far), want)
        del big_v


def test_empty():
    import torch
    z = torch.zeros
    cache = q4k.KVCache(*(z(2, 2, 16, 64, dtype=torch.float16, device="cuda") for _ in range(2)))
    i = lambda *s: z(s, dtype=torch.int32, device="cuda")  # noqa: E731
    for T, B in ((0, 0), (0, 2), (3, 0), (3, 2)):
        out = torch.full((T, 4, 64), 3.0, device="cuda")
        seqs = q4k.Sequences(i(B + 1), i(B), i(B, 2))
        q4k.attention(z(T, 4, 64, device="cuda"), cache, seqs, out=out)
        q4k.attention_tree(z(T, 4, 64, device="cuda"), cache, seqs, i(T, 1), out=out)
        assert (out == 3).all()


def test_offsets_out_of_order_stay_in_bounds():
    """Offsets that descend or pass T: rows hold anything, nothing else is touched."""
    import torch
    rng = rng_of(40)
    p = Paged(rng, [(40, 4), (3, 4), (9, 4)], 2, 64, 16, "f16")
    for bad in ([0, 9, 4, 12], [5, 2, 30, -4], [12, 8, 4, 0], [-9, 50, 60, 70], [0, 2 ** 31 - 1, -2 ** 31, 7]):
        p.offsets = np.array(bad, np.int32)
        cache, seqs = p.on_device()
        guard = torch.full((3, 12, 8, 64), 5.0, device="cuda")
        q = torch.randn(12, 8, 64, device="cuda")
        q4k.attention(q, cache, seqs, out=guard[1])
        q4k.attention_tree(q, cache, seqs, torch.ones(12, 1, dtype=torch.int32, device="cuda"), out=guard[1])
        torch.cuda.synchronize()
        assert (guard[0] == 5).all() and (guard[2] == 5).all()


def test_refusals():
    import torch
    z = lambda *s: torch.zeros(s, device="cuda")  # noqa: E731
    i = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    cache = q4k.KVCache(z(2, 2, 16, 64).half(), z(2, 2, 16, 64).half())
    seqs = q4k.Sequences(i(2), i(1), i(1, 2))
    q = z(3, 4, 64)
    with pytest.raises(q4k.Q4KError):
        q4k.attention(z(3, 3, 64), cache, seqs)
    with pytest.raises(ValueError, match="heads of 64"):
        q4k.attention(z(3, 4, 128), cache, seqs)
    with pytest.raises(ValueError, match="out"):
        q4k.attention(q, cache, seqs, out=q[:2])
    with pytest.raises(ValueError, match="contiguous"):
        q4k.attention(z(4, 3, 64).transpose(0, 1), cache, seqs)
    with pytest.raises(ValueError, match="mask"):
        q4k.attention_tree(q, cache, seqs, i(2, 1))
    with pytest.raises(TypeError, match="mask"):
        q4k.attention_tree(q, cache, seqs, i(3, 1).long())
    with pytest.raises(q4k.Q4KError):
        q4k.attention_tree(q, cache, seqs, i(3, 0))
    with pytest.raises(q4k.Q4KError):
        q4k.attention(z(1 + 3 * 256)[1:].view(3, 4, 64), cache, seqs)  # not 16-byte aligned
    with pytest.raises(ValueError, match="pages"):
        q4k.attention(q, cache, seqs._replace(pages=seqs.pages.cpu()))


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("sizes", [[(3000, 1)], [(3000, 8)], [(3000, 40)], [(200, 300), (0, 40)]])
def test_nan_keys_of_a_whole_part(sizes, kind):
    """Keys of NaN only over a stretch that one part of a split row may have to itself: NaN for every row."""
    rng = rng_of(41, len(sizes), sizes[0][1], TYPES.index(kind))
    p = Paged(rng, sizes, 2, 64, 16, kind)
    for page in p.table[0, :12]:
        p.k[int(page), 1] = float("nan")
    q = rng.standard_normal((p.T, 8, 64)).astype(np.float32)
    got = run(p, q, None).cpu().numpy()
    first = int(p.offsets[1])
    assert np.isnan(got[:first, 4:]).all()
    assert np.isfinite(got[:, :4]).all() and np.isfinite(got[first:]).all()


def test_values_of_every_size():
    """Weights over many powers of two: a maximum that rises from tile to tile (and falls) in small and
    large steps, in rows that are split and rows that are not."""
    rng = rng_of(42)
    for sizes in ([(1500, 1)], [(0, 300)], [(900, 50)]):
        for step in (0.01, 0.05, 0.4, -0.05):
            p = Paged(rng, sizes, 1, 64, 16, "f16")
            for b in range(len(sizes)):
                for j in range(int(p.lengths[b])):
                    p.k[int(p.table[b, j // 16]), :, j % 16, 0] = step * j / 8
            q = rng.standard_normal((p.T, 4, 64)).astype(np.float32)
            q[..., 0] = 4 + np.arange(4)
            cache, seqs = p.on_device()
            got = q4k.attention(to_dev(q), cache, seqs, 0.3).cpu().numpy()
            want, S, A = attention(p, q, 0.3)
            assert (np.abs(got - want) <= tolerance(p, S, A, int(p.lengths.max()))).all()


# (context, new tokens) of the sequences: with four query heads a key head tiles of 32, 64 and 128 rows, split along
# the keys and not, uneven rows, and sequences that fit none of their batch's tiles.
WIDE = {
    "32 rows": [(700, 8)],
    "32 rows, uneven": [(90, 1), (0, 15), (333, 8), (-3, 5), (0, 0), (1200, 7)],
    "64 rows": [(700, 16)],
    "64 rows, uneven": [(2, 30), (64, 1), (500, 17), (0, 3), (-2, 9)],
    "128 rows": [(900, 32)],
    "128 rows, uneven": [(40, 70), (300, 1), (0, 33), (0, 0), (65, 20)],
    "many tiles": [(13 * b % 70, 8) for b in range(70)],
    "many small": [(29 * b % 200, 1) for b in range(150)],
}


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("D", [48, 64, 96, 128, 256])
@pytest.mark.parametrize("name", WIDE)
def test_every_kernel(name, D, kind):
    """A table wide enough for a long context (which the choice of the kernel goes by), with and without a mask."""
    rng = rng_of(43, list(WIDE).index(name), D, TYPES.index(kind))
    sizes = WIDE[name]
    p = Paged(rng, sizes, 2, D, 16, kind, extra_rows=1, extra_cols=400)
    check(p, rng, 8)
    words = 3
    check(p, rng, 8, tree_mask(rng, sizes, words, 1), words)


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("n", [8, 16, 32])
def test_what_is_not_seen_in_every_kernel(n, kind):
    """As test_what_is_not_seen_never_reaches_a_row, for the tiles of 32, 64 and 128 rows."""
    import torch
    rng = rng_of(44, n, TYPES.index(kind))
    p = Paged(rng, [(300, n)], 2, 64, 16, kind, extra_cols=400)
    q = rng.standard_normal((n, 8, 64)).astype(np.float32)
    mask = tree_mask(rng, [(300, n)], 1)
    for m in (None, mask):
        clean = run(p, q, None, m).cpu().numpy()
        i = n // 2
        at = (int(p.table[0, (300 + i) // 16]), 1, (300 + i) % 16, 5)
        old = p.v[at].clone()
        p.v[at] = torch.tensor(float("nan")).to(p.v.dtype)
        got = run(p, q, None, m).cpu().numpy()
        p.v[at] = old
        see = np.arange(n) >= i if m is None else (m[:, 0] >> i & 1) == 1
        assert np.array_equal(got[~see], clean[~see]) and np.array_equal(got[:, :4], clean[:, :4])
        assert np.isnan(got[see][:, 4:, 5]).all()
        keep = np.arange(64) != 5
        assert np.array_equal(got[see][:, :, keep], clean[see][:, :, keep])


@pytest.mark.parametrize("page", [1, 2, 4, 8])
def test_small_pages_in_every_kernel(page):
    rng = rng_of(45, page)
    for sizes in ([(500, 8)], [(90, 16)], [(300, 40)], [(70, 1), (33, 1)]):
        for kind in ("f16", "e4m3"):
            check(Paged(rng, sizes, 1, 128, page, kind, extra_cols=6400 // page), rng, 4)


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("D", [80, 128, 208])
@pytest.mark.parametrize("page", [1, 64])
def test_many_tiles_of_few_rows(page, D, kind):
    """Enough row tiles for two workgroups on a CU, with contexts of many key tiles a wave (whose buffers are
    filled again and again), with and without a mask."""
    rng = rng_of(46, page, D, TYPES.index(kind))
    sizes = [(int(c), 1 + b % 3) for b, c in enumerate(rng.integers(0, 1500, 34))]
    p = Paged(rng, sizes, 2, D, page, kind, extra_rows=1)
    check(p, rng, 8)
    check(p, rng, 8, tree_mask(rng, sizes, 1, 1), 1)


@pytest.mark.parametrize("kind", TYPES)
def test_what_is_not_seen_by_many_tiles_of_few_rows(kind):
    import torch
    rng = rng_of(47, TYPES.index(kind))
    contexts = [0, 31, 300, 700] * 8
    p = Paged(rng, [(c, 3) for c in contexts], 2, 128, 16, kind)
    q = rng.standard_normal((96, 8, 128)).astype(np.float32)
    clean = run(p, q, None).cpu().numpy()
    for b, c in enumerate(contexts):
        p.v[int(p.table[b, (c + 1) // 16]), 1, (c + 1) % 16, 77] = torch.tensor(float("nan")).to(p.v.dtype)
    got = run(p, q, None).cpu().numpy()
    see = np.arange(96) % 3 >= 1
    assert np.array_equal(got[~see], clean[~see]) and np.array_equal(got[:, :4], clean[:, :4])
    assert np.isnan(got[see][:, 4:, 77]).all()
    keep = np.arange(128) != 77
    assert np.array_equal(got[see][:, :, keep], clean[see][:, :, keep])


@pytest.mark.parametrize("kind", TYPES)
def test_as_many_tiles_as_workgroups(kind):
    """Every workgroup takes one row tile, the most keys first: sequences of one length, of every length, without
    new tokens and without a context, more than are looked through at once."""
    rng = rng_of(48, TYPES.index(kind))
    for B in (65, 300):
        for n, longest in ((1, 400), (3, 1)):
            sizes = [(int(c), int(rng.integers(0, n + 1))) for c in rng.integers(0, longest // 2 + 1, B)]
            check(Paged(rng, sizes, 8, 32, 16, kind, extra_rows=1), rng, 16)
    check(Paged(rng, [(70, 2)] * 150, 8, 16, 16, kind), rng, 8)
    check(Paged(rng, [(0, 900), (300, 0), (0, 0), (17, 500)], 8, 16, 16, kind), rng, 32)
    check(Paged(rng, [(int(c), 20) for c in rng.integers(0, 90, 130)], 8, 16, 16, kind), rng, 64)
    check(Paged(rng, [(5, 1000)], 8, 16, 16, kind), rng, 32)
