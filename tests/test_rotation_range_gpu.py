"""The rotation (include/q4k_layer.h) at the farthest positions, against angles of the exact product."""
from fractions import Fraction

import numpy as np
import pytest

import gguf_q4_dequant_amd as q4k
from tests.gpu_helpers import to_dev
from tests.layer_reference import rng_of

pytestmark = pytest.mark.gpu

TWO_PI = 2 * (Fraction(np.pi) + Fraction(1.2246467991473532e-16))  # pi in two doubles: 106 bits


def angle(position, f):
    """position * f less its whole turns, from the exact product."""
    x = Fraction(int(position)) * Fraction(float(f))
    return float(x - TWO_PI * round(x / TWO_PI))


@pytest.mark.parametrize("interleaved", [False, True], ids=["halves", "interleaved"])
def test_far_positions(interleaved):
    """A position of 31 bits times a frequency of 24 has 55: rounded to a double it is off by 2^-54 of
    itself, 2^-23 where the frequency is 1 and 2^-12 where it is 2000."""
    import torch
    rng = rng_of(95, int(interleaved))
    D, T = 128, 96
    f = np.exp(rng.uniform(np.log(0.5), np.log(4000), D // 2)).astype(np.float32)
    f[:4] = np.nextafter(np.float32(1), np.float32(0)), 1, 4.0, 1e-3
    positions = (2 ** 31 - 1 - 2 * rng.integers(0, 2 ** 20, T)).astype(np.int32)
    positions[:3] = 2 ** 31 - 1, -2 ** 31, -2 ** 31 + 1
    q = rng.standard_normal((T, 1, D)).astype(np.float32)
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    cache = q4k.KVCache(*(torch.zeros(1, 1, 128, D, dtype=torch.float16, device="cuda") for _ in range(2)))
    got = q4k.kv_append(to_dev(q), to_dev(q), cache, q4k.Sequences(i32(0, T), i32(T), i32(0).view(1, 1)),
                        rotation=q4k.Rotation(to_dev(f), interleaved), q=to_dev(q), positions=to_dev(positions))
    a = np.array([[angle(p, x) for x in f] for p in positions])
    c, s = np.cos(a)[:, None], np.sin(a)[:, None]
    at = (slice(0, D, 2), slice(1, D, 2)) if interleaved else (slice(0, D // 2), slice(D // 2, D))
    u, w = q[..., at[0]].astype(np.float64), q[..., at[1]].astype(np.float64)
    got = got.cpu().numpy()
    # the angle's rounding to float32 (2^-25 of half a turn), cos and sin (2^-23 each, two steps of float32),
    # two products and a sum (2^-24 each of the pair's size)
    tol = (2.0 ** -25 * np.pi + 2 * 2.0 ** -23 + 3 * 2.0 ** -24) * np.hypot(u, w)
    assert (np.abs(got[..., at[0]] - (u * c - w * s)) <= tol).all()
    assert (np.abs(got[..., at[1]] - (w * c + u * s)) <= tol).all()
