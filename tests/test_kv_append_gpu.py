"""New tokens' keys and values in the paged cache, and the rotation
(include/q4k_layer.h), against 64 bits."""
import numpy as np
import pytest

import gguf_q4_dequant_amd as q4k
from tests.gpu_helpers import to_dev
from tests.layer_reference import TYPES, Paged, rng_of, rotation

pytestmark = pytest.mark.gpu

# float32 work before the last rounding, relative to the size of a rotated pair: the
# norm's factor (2^-22: sum of up to 256 squares in float32, root, quotient) and its two
# products, cos and sin (2^-22 each), two products and a sum, the division by the scale.
WORK = 2.0 ** -20
HALF_STEP = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8, "e4m3": 2.0 ** -4}
LEAST = {"f16": 2.0 ** -25, "bf16": 2.0 ** -134, "e4m3": 2.0 ** -10}  # half a step below the normal numbers


def check(p, rng, q_heads, norm, R, interleaved, positions=None, q_given=True, extra=0):
    import torch
    D, Hk, T = p.D, p.kv_heads, p.T
    k, v, q = (rng.standard_normal((T, h, D)).astype(np.float32) for h in (Hk, Hk, q_heads))
    k[..., 0] *= 20
    wq, wk = ((rng.random(D) + 0.5).astype(np.float32) for _ in range(2)) if norm else (None, None)
    f = (10000.0 ** (-np.arange(R // 2) / max(R // 2, 1))).astype(np.float32) if R else None
    cache, seqs = p.on_device()
    dev = lambda a: None if a is None else to_dev(a)  # noqa: E731
    sentinel = torch.full((T, q_heads, D), 7.25, device="cuda")
    out = q4k.kv_append(dev(k), dev(v), cache, seqs, rotation=None if f is None else q4k.Rotation(to_dev(f), interleaved),
                        q=dev(q) if q_given else None, positions=dev(positions), q_norm=dev(wq), k_norm=dev(wk),
                        eps=1e-5, q_out=sentinel if q_given else None)
    n = int(p.offsets[-1])
    seq = np.searchsorted(p.offsets[1:], np.arange(n), side="right")
    index = p.lengths[seq] - p.offsets[seq + 1] + np.arange(n)
    pos = index if positions is None else positions[:n]
    if q_given:
        assert out is sentinel
        want, size = rotation(q[:n], wq, 1e-5, pos, f, interleaved)
        got = out.cpu().numpy()
        assert (np.abs(got[:n] - want) <= WORK * size).all()
        assert (got[n:] == 7.25).all()
    else:
        assert out is None
    raw = torch.uint8 if p.kind == "e4m3" else torch.int16
    kk, ksize = rotation(k[:n], wk, 1e-5, pos, f, interleaved)
    written = np.zeros(p.k.shape[:1] + p.k.shape[2:3], bool)
    for name, got, start, want, size, scale in (("k", cache.k, p.k, kk, ksize, p.k_scale),
                                                ("v", cache.v, p.v, v[:n].astype(np.float64), np.abs(v[:n]), p.v_scale)):
        got = got.cpu()
        g = got.double().numpy()
        for i in range(n):
            j, b = int(index[i]), int(seq[i])
            col = j // p.page
            page = p.table[b, col] if j >= 0 and col < p.table.shape[1] else -1
            if not 0 <= page < p.pool:
                continue
            written[page, j % p.page] = True
            w, s = want[i] / scale, size[i] / scale
            if p.kind == "e4m3":
                w, s = np.clip(w, -448, 448), np.minimum(s, 448 * 2)
            off = np.abs(g[page, :, j % p.page] - w)
            assert (off <= HALF_STEP[p.kind] * (np.abs(w) + WORK * s) + WORK * s + LEAST[p.kind]).all(), (name, i)
        # every other place is as it was, bit for bit
        keep = ~np.broadcast_to(written[:, None, :, None], got.shape)
        assert (got.view(raw).numpy()[keep] == start.view(raw).numpy()[keep]).all()


SETS = {
    "one token": [(1000, 1)],
    "first token": [(0, 1)],
    "prompts": [(0, 37), (0, 1), (0, 130)],
    "ragged": [(5, 3), (0, 0), (64, 1), (31, 18), (0, 2), (0, 0)],
    "many": [(3 * b, 1 + b % 2) for b in range(150)],
}


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("interleaved", [False, True], ids=["halves", "interleaved"])
@pytest.mark.parametrize("name", SETS)
def test_append(name, interleaved, kind):
    rng = rng_of(10, list(SETS).index(name), int(interleaved), TYPES.index(kind))
    scales = (0.05, 0.07) if kind == "e4m3" else (1.0, 1.0)
    p = Paged(rng, SETS[name], 2, 64, 16, kind, *scales, new_empty=True, extra_rows=3)
    check(p, rng, 6, False, 64, interleaved)


@pytest.mark.parametrize("interleaved", [False, True], ids=["halves", "interleaved"])
@pytest.mark.parametrize("D,R", [(16, 16), (32, 24), (48, 48), (80, 32), (80, 80), (96, 96), (128, 128), (128, 8),
                                 (160, 160), (192, 64), (256, 256), (64, 0)])
def test_head_sizes_partial_rotation_and_norms(D, R, interleaved):
    rng = rng_of(11, D, R, int(interleaved))
    p = Paged(rng, [(9, 4), (0, 7)], 3, D, 8, "f16", new_empty=True)
    check(p, rng, 3, True, R, interleaved)


@pytest.mark.parametrize("page", [1, 2, 64, 1024])
def test_page_sizes(page):
    rng = rng_of(12, page)
    check(Paged(rng, [(70, 9), (1, 70)], 2, 32, page, "bf16", new_empty=True), rng, 2, True, 32, False)


@pytest.mark.parametrize("scales", [(1.0, 1.0), (3.0, 0.01)])
@pytest.mark.parametrize("kind", TYPES)
def test_scales(kind, scales):
    rng = rng_of(13, TYPES.index(kind), int(scales[0]))
    check(Paged(rng, [(3, 20)], 2, 64, 16, kind, *scales, new_empty=True), rng, 4, False, 64, False)


def test_given_and_far_positions():
    rng = rng_of(14)
    p = Paged(rng, [(3, 5), (40, 4)], 1, 64, 16, "f16", new_empty=True)
    pos = np.array([0, 131072, 1000003, 2 ** 24 + 1, 2 ** 31 - 1, -1, -70000, 5, 5], np.int32)
    check(p, rng, 2, True, 64, True, positions=pos)


def test_without_queries_or_rotation():
    rng = rng_of(15)
    p = Paged(rng, [(3, 5), (0, 4)], 2, 64, 16, "f16", new_empty=True)
    check(p, rng, 2, False, 0, False, q_given=False)
    check(p, rng, 2, False, 0, False)
    check(p, rng, 16, True, 0, False)


def test_tokens_without_a_place_are_not_stored():
    rng = rng_of(16)
    p = Paged(rng, [(10, 6), (5, 20), (0, 3), (-4, 6)], 2, 32, 8, "f16", new_empty=True)
    p.table[0, 1] = -1            # a missing page
    p.table[1, 2] = p.pool        # behind the pool
    p.table[2, 0] = -2 ** 31
    p.lengths[1] = 60             # the new tokens behind the table's last page
    check(p, rng, 2, False, 32, False)


def test_e4m3_saturates_and_keeps_nan():
    import torch
    k = torch.tensor([447.9, 449.0, 1e9, -1e9, float("inf"), -float("inf"), float("nan"), 0.0009, 0.0010, -0.0, 464.0,
                      465.0, 17.0, 19.0, 2.0 ** -9, 2.0 ** -6], device="cuda").view(1, 1, 16)
    cache = q4k.KVCache(*(torch.zeros(1, 1, 1, 16, dtype=torch.float8_e4m3fn, device="cuda") for _ in range(2)))
    i = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    q4k.kv_append(k, k, cache, q4k.Sequences(i(0, 1), i(1), i(0).view(1, 1)))
    want = k.clamp(-448, 448).cpu().to(torch.float8_e4m3fn)
    for got in (cache.k, cache.v):
        g, w = got.cpu().float().flatten(), want.float().flatten()
        assert torch.equal(torch.isnan(g), torch.isnan(w)) and torch.equal(g[~torch.isnan(w)], w[~torch.isnan(w)])


def test_rounding_is_torchs():
    """f16 and bf16: to the nearest, ties to even, subnormal numbers and overflow as torch rounds them."""
    import torch
    x = torch.randn(64, 1, 64, device="cuda") * torch.logspace(-9, 6, 64, device="cuda")[:, None, None]
    i = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    for dtype in (torch.float16, torch.bfloat16):
        cache = q4k.KVCache(*(torch.zeros(1, 1, 64, 64, dtype=dtype, device="cuda") for _ in range(2)))
        q4k.kv_append(x, x, cache, q4k.Sequences(i(0, 64), i(64), i(0).view(1, 1)))
        assert torch.equal(cache.k[0, 0], x[:, 0].to(dtype)) and torch.equal(cache.v[0, 0], x[:, 0].to(dtype))


def test_in_place_queries():
    import torch
    rng = rng_of(17)
    p = Paged(rng, [(4, 9)], 2, 128, 16, "f16", new_empty=True)
    cache, seqs = p.on_device()
    k, q = torch.randn(9, 2, 128, device="cuda"), torch.randn(9, 8, 128, device="cuda")
    rot = q4k.Rotation(torch.rand(64, device="cuda"))
    want = q4k.kv_append(k, k, cache, seqs, rotation=rot, q=q)
    got = q4k.kv_append(k, k, cache, seqs, rotation=rot, q=q, q_out=q)
    assert got is q and torch.equal(got, want)


def test_offsets_past_32_bits():
    """The last page of a pool of more than 2^32 elements."""
    import torch
    page, heads, D = 1024, 8, 128
    pages = (1 << 32) // (page * heads * D) + 3
    pool = torch.zeros(pages, heads, page, D, dtype=torch.float8_e4m3fn, device="cuda")
    cache = q4k.KVCache(pool, pool)
    i = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    k = torch.randn(2, heads, D, device="cuda")
    q4k.kv_append(k, k, cache, q4k.Sequences(i(0, 2), i(page), i(pages - 1).view(1, 1)))
    assert torch.equal(pool[pages - 1, :, page - 2:].float(), k.transpose(0, 1).to(torch.float8_e4m3fn).float())
    assert int(pool.view(torch.uint8)[:pages - 1].amax()) == 0 and int(pool.view(torch.uint8)[pages - 1, :, :page - 2].amax()) == 0


def test_empty():
    import torch
    z = torch.zeros
    cache = q4k.KVCache(*(z(2, 2, 16, 64, dtype=torch.float16, device="cuda") for _ in range(2)))
    i = lambda *s: z(s, dtype=torch.int32, device="cuda")  # noqa: E731
    for T, B in ((0, 0), (0, 2), (3, 0)):
        q = torch.full((T, 4, 64), 3.0, device="cuda")
        out = q4k.kv_append(z(T, 2, 64, device="cuda"), z(T, 2, 64, device="cuda"), cache, q4k.Sequences(i(B + 1), i(B), i(B, 2)), q=q, q_out=q)
        assert (out == 3).all()


def test_refusals():
    import torch
    z = lambda *s, **k: torch.zeros(s, device="cuda", **k)  # noqa: E731
    i = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    cache = q4k.KVCache(z(2, 2, 16, 64).half(), z(2, 2, 16, 64).half())
    seqs = q4k.Sequences(i(2), i(1), i(1, 2))
    k = z(3, 2, 64)
    with pytest.raises(ValueError, match="heads of 64"):
        q4k.kv_append(z(3, 4, 64), z(3, 4, 64), cache, seqs)
    with pytest.raises(ValueError, match="v must be"):
        q4k.kv_append(k, k[:2], cache, seqs)
    with pytest.raises(ValueError, match="q must be"):
        q4k.kv_append(k, k, cache, seqs, q=z(3, 3, 64))
    with pytest.raises(ValueError, match="q must be"):
        q4k.kv_append(k, k, cache, seqs, q=z(2, 4, 64))
    with pytest.raises(ValueError, match="q_out"):
        q4k.kv_append(k, k, cache, seqs, q_out=k)
    with pytest.raises(ValueError, match="positions"):
        q4k.kv_append(k, k, cache, seqs, positions=i(2))
    with pytest.raises(ValueError, match="q_norm"):
        q4k.kv_append(k, k, cache, seqs, q_norm=z(32))
    with pytest.raises(ValueError, match="lengths"):
        q4k.kv_append(k, k, cache, q4k.Sequences(i(2), i(2), i(1, 2)))
    with pytest.raises(ValueError, match="offsets"):
        q4k.kv_append(k, k, cache, q4k.Sequences(i(1), i(1), i(1, 2)))
    with pytest.raises(TypeError, match="lengths"):
        q4k.kv_append(k, k, cache, q4k.Sequences(i(2), i(1).long(), i(1, 2)))
    with pytest.raises(q4k.Q4KError):
        q4k.kv_append(k, k, cache, seqs, rotation=q4k.Rotation(z(6)))
    with pytest.raises(q4k.Q4KError):
        q4k.kv_append(k, k, cache._replace(k_scale=0.0), seqs)
    odd = q4k.KVCache(z(2, 2, 12, 64).half(), z(2, 2, 12, 64).half())
    with pytest.raises(q4k.Q4KError):
        q4k.kv_append(k, k, odd, seqs)
