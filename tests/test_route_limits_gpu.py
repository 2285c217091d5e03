"""Routing by scores far below what float32 holds: sigmoids of very low logits keep
their order and their shares as long as a double holds them (down to about -745)."""
import numpy as np
import pytest

import gguf_q4_dequant_amd as q4k
from tests.gpu_helpers import to_dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M", [1, 40])
@pytest.mark.parametrize("bias", [False, True])
def test_sigmoids_of_very_low_logits(M, bias):
    E, k = 70, 4
    z = np.full((M, E), -1000.0, np.float32)
    place = np.array([69, 3, 64, 30])                       # best first
    z[:, place] = np.array([-705.5, -711.25, -720.0, -735.0], np.float32)
    r = q4k.moe_route(to_dev(z), k, bias=to_dev(np.zeros(E, np.float32)) if bias else None, sigmoid=True)
    assert np.array_equal(r.expert.cpu().numpy(), np.tile(place, (M, 1)).astype(np.int32))
    # s = exp(z) / (1 + exp(z)), the quotient's denominator 1 to the last bit
    share = np.exp(z[0, place].astype(np.float64) + 705.5)
    want = share / share.sum()
    # a subnormal double is off by half its step, 2^-1075, the exponential by an ulp
    # or two; the share in float32 by 2^-24, or half of its own smallest step
    off = (2.0 ** -1074 * np.exp(705.5)) * 2 / share.sum() + 2.0 ** -24 * want + 2.0 ** -149
    got = r.weight.cpu().numpy().astype(np.float64)
    assert np.all(np.abs(got - want) <= off), (got, want)


def test_a_single_very_low_score_is_the_whole_share():
    z = np.full((20, 9), -np.inf, np.float32)
    z[:, 5] = np.linspace(-744.0, -700.0, 20)
    r = q4k.moe_route(to_dev(z), 2, sigmoid=True)
    assert np.array_equal(r.expert.cpu().numpy(), np.tile([5, -1], (20, 1)))
    assert np.array_equal(r.weight.cpu().numpy(), np.tile(np.float32([1, 0]), (20, 1)))
