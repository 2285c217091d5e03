"""Attention over values near the ends of their type's range, and under scales near the ends of
float32's (include/q4k_layer.h), against 64 bits: what is finite stays finite and exact."""
import numpy as np
import pytest

import gguf_q4_dequant_amd as q4k
from tests.gpu_helpers import to_dev
from tests.layer_reference import TYPES, Paged, attention, rng_of, tolerance

pytestmark = pytest.mark.gpu

# Four query heads a key head: tiles of 16, 32, 64 and 128 rows, split along the keys and not.
SIZES = {"one key": [(0, 1)], "16 rows": [(700, 1), (3, 2)], "32 rows": [(700, 8)], "64 rows": [(700, 16)],
         "128 rows": [(900, 40)], "prompts": [(0, 90), (0, 300)], "many tiles": [(9 * b % 70, 1) for b in range(130)]}


def run(p, q, scale):
    cache, seqs = p.on_device()
    got = q4k.attention(to_dev(q), cache, seqs, scale).cpu().numpy()
    want, S, A = attention(p, q, scale)
    return got, want, tolerance(p, S, A, int(p.lengths.max()))


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("name", SIZES)
def test_values_near_the_types_largest(name, kind):
    """Values of the type's largest size, of one sign in half of the dimensions: the weighted sums in front of
    the division are as large as they get."""
    import torch
    rng = rng_of(80, list(SIZES).index(name), TYPES.index(kind))
    p = Paged(rng, SIZES[name], 2, 64, 16, kind, extra_cols=400)
    largest = torch.finfo(p.v.dtype).max
    sign = torch.from_numpy(np.sign(rng.standard_normal(p.v.shape)))
    sign[..., ::2] = 1
    p.v = torch.where(p.v.double().isfinite(), sign * largest, p.v.double()).to(p.v.dtype)
    q = rng.standard_normal((p.T, 8, 64)).astype(np.float32)
    got, want, tol = run(p, q, 0.125)
    assert np.isfinite(got).all()
    assert (np.abs(got.astype(np.float64) - want) <= tol).all()


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("v_scale", [2.0 ** -120, 2.0 ** 120])
@pytest.mark.parametrize("name", SIZES)
def test_scales_near_float32s_ends(name, v_scale, kind):
    """Outputs are normal numbers (2^-120 of values near 1), so they lose nothing beside one more rounding."""
    rng = rng_of(81, list(SIZES).index(name), int(v_scale > 1), TYPES.index(kind))
    p = Paged(rng, SIZES[name], 2, 64, 16, kind, extra_cols=400)
    p.v_scale = v_scale
    q = rng.standard_normal((p.T, 8, 64)).astype(np.float32)
    got, want, tol = run(p, q, 0.125)
    assert (np.abs(got.astype(np.float64) - want) <= tol + 2.0 ** -24 * np.abs(want) + 2.0 ** -149).all()
