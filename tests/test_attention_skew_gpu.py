"""Batches with as many row tiles as workgroups and contexts of very different lengths: one sequence
with most of the batch's keys, in tiles of 16, 32, 64 and 128 rows, against 64 bits."""
import numpy as np
import pytest

import gguf_q4_dequant_amd as q4k
from tests.gpu_helpers import to_dev
from tests.layer_reference import Paged, attention, rng_of, tolerance

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
