"""Batches with as many row tiles as workgroups and contexts of very different lengths: one sequence
with most of the batch's keys, in tiles of 16, 32, 64 and 128 rows, against 64 bits."""
import numpy as np
import pytest

import gguf_q4_dequant_amd as q4k
from tests.gpu_helpers import to_dev
from tests.layer_reference import TYPES, Paged, attention, rng_of, tolerance, tree_mask

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["f16", "e4m3"])
@pytest.mark.parametrize("tokens", [1, 8, 16, 40])
def test_one_long_context_among_short_ones(tokens, kind):
    """Four query heads a key head, eight key heads: 64 sequences or more are one row tile a workgroup."""
    rng = rng_of(140, tokens, kind == "e4m3")
    sizes = [(int(c), tokens) for c in rng.integers(0, 40, 66)]
    sizes[17] = (9000, tokens)
    sizes[40] = (1500, tokens)
    p = Paged(rng, sizes, 8, 16, 16, kind)
    q = rng.standard_normal((p.T, 32, 16)).astype(np.float32)
    cache, seqs = p.on_device()
    got = q4k.attention(to_dev(q), cache, seqs).cpu().numpy()
    # 64 bits for the two long sequences and two short ones (a row's others say nothing more)
    keep = [17, 40, 0, 65]
    p.sizes = [sizes[b] for b in keep]
    rows = np.concatenate([np.arange(p.offsets[b], p.offsets[b + 1]) for b in keep])
    p.table, p.lengths = p.table[keep], p.lengths[keep]
    p.offsets = np.arange(len(keep) + 1) * tokens
    want, S, A = attention(p, q[rows], 0.25)
    off, tol = np.abs(got[rows] - want), tolerance(p, S, A, 9040)
    assert (off <= tol).all(), float((off / tol).max())


def test_many_sequences():
    """Many more sequences than are looked through at once, in the cache and in the attention."""
    rng = rng_of(141)
    B = 5000
    sizes = [(int(c), 1) for c in rng.integers(0, 6, B)]
    p = Paged(rng, sizes, 1, 16, 8, "f16")
    q = rng.standard_normal((B, 2, 16)).astype(np.float32)
    cache, seqs = p.on_device()
    got = q4k.attention(to_dev(q), cache, seqs).cpu().numpy()
    want, S, A = attention(p, q, 0.25)
    assert (np.abs(got - want) <= tolerance(p, S, A, 7)).all()
    k = rng.standard_normal((B, 1, 16)).astype(np.float32)
    q4k.kv_append(to_dev(k), to_dev(k), cache, seqs)
    stored = cache.k.cpu().float().numpy()
    for b in range(B):
        j = int(p.lengths[b]) - 1
        assert np.array_equal(stored[p.table[b, j // 8], 0, j % 8], k[b, 0].astype(np.float16).astype(np.float32))


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("B,longs", [(65, (5000,)), (200, (4200, 6100, 90)), (256, (7000, 7000)), (257, (6000,)), (1000, (6000,))])
def test_uneven_batches(B, longs, kind):
    """A row tile a workgroup, or the line cut where the longest context is far above the others' (up to 256
    sequences); sequences without new tokens and without a context; causal and with a mask."""
    rng = rng_of(142, B, TYPES.index(kind))
    sizes = [(int(c), int(n)) for c, n in zip(rng.integers(0, 30, B), rng.integers(0, 3, B))]
    for c in longs:
        sizes[int(rng.integers(B))] = (c, 2)
    p = Paged(rng, sizes, 8, 16, 16, kind, extra_rows=1)
    q = rng.standard_normal((p.T, 16, 16)).astype(np.float32)
    cache, seqs = p.on_device()
    out = to_dev(np.full(q.shape, 7.25, np.float32))
    mask = tree_mask(rng, sizes, 1, 1)
    for m in (None, mask):
        if m is None:
            q4k.attention(to_dev(q), cache, seqs, out=out)
        else:
            q4k.attention_tree(to_dev(q), cache, seqs, to_dev(m.view(np.int32)), out=out)
        got = out.cpu().numpy()
        assert (got[-1] == 7.25).all()
        with np.errstate(invalid="ignore"):
            want, S, A = attention(p, q, 0.25, m, 1)
        off, tol = np.abs(got - want)[:-1], tolerance(p, S, A, max(longs))[:-1]
        assert (off <= tol).all(), float((off / tol).max())


def test_uneven_batches_in_a_graph():
    """Whether the line is cut is found on the device: lengths that change between replays."""
    import torch
    rng = rng_of(143)
    p = Paged(rng, [(6000, 1)] + [(int(c), 1) for c in rng.integers(0, 60, 79)], 8, 64, 16, "f16")
    cache, seqs = p.on_device()
    q = to_dev(rng.standard_normal((80, 16, 64)).astype(np.float32))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        q4k.attention(q, cache, seqs)
        side.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            outs = [q4k.attention(q, cache, seqs) for _ in range(2)]
    torch.cuda.synchronize()
    for first in (6001, 40, 3000, 6001, 0, 4500):
        seqs.lengths[0] = first
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        want = q4k.attention(q, cache, seqs)
        assert all(torch.equal(o, want) for o in outs), first
        p.lengths[0] = first
        with np.errstate(invalid="ignore"):
            exact, S, A = attention(p, q.cpu().numpy(), 0.125)
        assert (np.abs(want.cpu().numpy() - exact) <= tolerance(p, S, A, 6001)).all(), first


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("D", [48, 128, 256])
def test_uneven_batches_of_every_kernel(D, kind):
    """The kernels of few rows for other head sizes, with NaN keys over a stretch that one part has to itself."""
    rng = rng_of(144, D, TYPES.index(kind))
    sizes = [(int(c), 1 + b % 2) for b, c in enumerate(rng.integers(0, 50, 70))]
    sizes[33] = (6000, 2)
    sizes[50] = (4700, 1)
    p = Paged(rng, sizes, 8, D, 32, kind)
    q = rng.standard_normal((p.T, 16, D)).astype(np.float32)
    cache, seqs = p.on_device()
    got = q4k.attention(to_dev(q), cache, seqs).cpu().numpy()
    keep = [33, 50, 0, 69]
    rows = np.concatenate([np.arange(p.offsets[b], p.offsets[b + 1]) for b in keep])
    few = Paged.__new__(Paged)
    few.__dict__.update(p.__dict__)
    few.sizes = [sizes[b] for b in keep]
    few.table, few.lengths = p.table[keep], p.lengths[keep]
    few.offsets = np.concatenate([[0], np.cumsum([n for _, n in few.sizes])])
    want, S, A = attention(few, q[rows], D ** -0.5)
    off, tol = np.abs(got[rows] - want), tolerance(few, S, A, 6002)
    assert (off <= tol).all(), float((off / tol).max())
    for page in p.table[50, :16]:
        p.k[int(page), 3] = float("nan")
    cache, seqs = p.on_device()
    bad = q4k.attention(to_dev(q), cache, seqs).cpu().numpy()
    hit = np.zeros(bad.shape, bool)
    hit[p.offsets[50]:p.offsets[51], 6:8] = True
    assert np.isnan(bad[hit]).all() and np.array_equal(bad[~hit], got[~hit])


def test_uneven_batches_with_offsets_out_of_order():
    """Rows hold anything, and nothing else is touched; the next call is right."""
    import torch
    rng = rng_of(145)
    p = Paged(rng, [(6000, 1)] + [(int(c), 1) for c in rng.integers(0, 60, 79)], 8, 16, 16, "f16")
    cache, seqs = p.on_device()
    q = to_dev(rng.standard_normal((80, 16, 16)).astype(np.float32))
    want = q4k.attention(q, cache, seqs)
    guard = torch.full((3, *q.shape), 5.0, device="cuda")
    for bad in (seqs.offsets.flip(0), seqs.offsets * 7 - 90, seqs.offsets[torch.randperm(81)], seqs.offsets % 9):
        q4k.attention(q, cache, seqs._replace(offsets=bad.contiguous()), out=guard[1])
        torch.cuda.synchronize()
        assert (guard[0] == 5).all() and (guard[2] == 5).all()
        assert torch.equal(q4k.attention(q, cache, seqs), want)
