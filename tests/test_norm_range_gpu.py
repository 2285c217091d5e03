"""The norms (include/q4k_layer.h) of rows and heads near the ends of float32's range, against 64 bits."""
import numpy as np
import pytest

import gguf_q4_dequant_amd as q4k
from tests.gpu_helpers import to_dev
from tests.layer_reference import rng_of, rotation

pytestmark = pytest.mark.gpu

SIZES = [2.0 ** -140, 1e-38, 1e-30, 1e-20, 1e-10, 1.0, 1e10, 1e20, 1e30, 1e37]


@pytest.mark.parametrize("eps", [0.0, 1e-6])
@pytest.mark.parametrize("N", [5, 300, 5000])
def test_norm_of_rows_of_every_size(N, eps):
    """The factor is beyond float32 for rows below 2^-128, and loses bits for rows above 2^126."""
    rng = rng_of(90, N, int(eps > 0))
    x = (rng.standard_normal((len(SIZES), N)) * np.array(SIZES)[:, None]).astype(np.float32)
    w = (0.5 + rng.random(N)).astype(np.float32)
    t = x.astype(np.float64)
    want = t / np.sqrt((t * t).mean(1, keepdims=True) + eps) * w
    got = q4k.rms_norm(to_dev(x), to_dev(w), eps).cpu().numpy()
    # the factor and two products rounded, each by 2^-24, or by half of the least subnormal number (times a weight of up to 1.5)
    assert (np.abs(got - want) <= 4 * 2.0 ** -24 * np.abs(want) + 2.0 ** -148).all()


@pytest.mark.parametrize("interleaved", [False, True], ids=["halves", "interleaved"])
@pytest.mark.parametrize("D", [16, 80, 128, 256])
@pytest.mark.parametrize("eps", [0.0, 1e-6])
def test_norm_of_heads_of_every_size(D, eps, interleaved):
    """As the rows of rms_norm: what a head's values are squared to fits float32 only from 1e-19 to 1e18."""
    import torch
    rng = rng_of(91, D, int(eps > 0), int(interleaved))
    T, page = len(SIZES), 16
    q, k = ((rng.standard_normal((T, h, D)) * np.array(SIZES)[:, None, None]).astype(np.float32) for h in (4, 2))
    wq, wk = ((0.5 + rng.random(D)).astype(np.float32) for _ in range(2))
    f = (10000.0 ** (-np.arange(D // 2) / (D // 2))).astype(np.float32)
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    cache = q4k.KVCache(*(torch.zeros(1, 2, page, D, dtype=torch.bfloat16, device="cuda") for _ in range(2)))
    seqs = q4k.Sequences(i32(0, T), i32(T), i32(0).view(1, 1))
    got = q4k.kv_append(to_dev(k), to_dev(k), cache, seqs, rotation=q4k.Rotation(to_dev(f), interleaved), q=to_dev(q),
                        q_norm=to_dev(wq), k_norm=to_dev(wk), eps=eps).cpu().numpy()
    want, size = rotation(q, wq, eps, np.arange(T), f, interleaved)
    # the factor, two products, cos and sin (2^-22 each), two products and a sum, as in the tests of the append
    assert (np.abs(got - want) <= 2.0 ** -20 * size + 2.0 ** -146).all()
    want, size = rotation(k, wk, eps, np.arange(T), f, interleaved)
    stored = cache.k[0].double().cpu().numpy().transpose(1, 0, 2)[:T]
    assert (np.abs(stored - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -19 * size + 2.0 ** -132).all()
