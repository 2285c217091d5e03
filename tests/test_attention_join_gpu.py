"""Rows in more parts than a wave has lanes, joined by a second launch that has many rows (a wave each), of
tiles of 32, 64 and 128 rows; and joined by whole workgroups where there are few."""
import numpy as np
import pytest

import gguf_q4_dequant_amd as q4k
from tests.gpu_helpers import to_dev
from tests.layer_reference import Paged, attention, rng_of, tolerance

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [64, 80])
@pytest.mark.parametrize("tokens,others", [(2, 64), (4, 32), (8, 16), (2, 10), (8, 3)])
def test_a_row_of_many_parts(tokens, others, D):
    """16 query heads on one key head: 20000 keys are cut into 78 parts or more."""
    rng = rng_of(130, tokens, others, D)
    sizes = [(int(rng.integers(0, 40)), tokens) for _ in range(others)]
    sizes.insert(others // 2, (20000, tokens))
    p = Paged(rng, sizes, 1, D, 64, "f16")
    q = rng.standard_normal((p.T, 16, D)).astype(np.float32)
    cache, seqs = p.on_device()
    got = q4k.attention(to_dev(q), cache, seqs).cpu().numpy()
    want, S, A = attention(p, q, D ** -0.5)
    off, tol = np.abs(got - want), tolerance(p, S, A, 20008)
    assert (off <= tol).all(), float((off / tol).max())
