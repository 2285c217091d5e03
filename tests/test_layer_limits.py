"""Limits of the norm, cache and attention entry points that are told without a GPU."""
import os

import numpy as np
import pytest

import gguf_q4_dequant_amd as q4k
from tests.test_layer_abi import A, CALLS, cache, make, seqs


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(q4k.LIBRARY_PATH):
        from gguf_q4_dequant_amd import build
        build.build()
    return q4k.library()


@pytest.mark.parametrize("what", CALLS)
@pytest.mark.parametrize("name", ["k_scale", "v_scale"])
def test_scales_whose_reciprocal_is_infinite(lib, what, name):
    """The append multiplies by 1 / scale: below 2^-128 that is infinite, and zeros would be stored as NaN."""
    call = make(lib, what)
    for scale in (2.0 ** -149, 2.0 ** -130, 2.0 ** -128):
        assert call(c=cache(**{name: scale})) == q4k.ERR_BAD_DIM, scale
    for scale in (np.nextafter(np.float32(2.0 ** -128), np.float32(1)), 2.0 ** -127, 2.0 ** -126, float(np.finfo(np.float32).max)):
        assert call(T=0, c=cache(**{name: float(scale)})) == q4k.OK, scale


def test_heads_of_queries_that_are_not_given(lib):
    """q_heads is looked at where q is given, and only there."""
    call = make(lib, "append")
    for heads in (0, 1, 3, 5, -1, 1 << 29):
        assert call(q=None, q_out=None, k=None, T=4, q_heads=heads) == q4k.ERR_NULL, heads  # (of k)
        assert call(q=None, q_out=None, T=0, q_heads=heads) == q4k.OK, heads
    for heads in (0, 1, 3, 5, -1, 1 << 29):
        assert call(k=None, T=4, q_heads=heads) == q4k.ERR_BAD_DIM, heads
    assert call(k=None, T=4, q_heads=4) == q4k.ERR_NULL
