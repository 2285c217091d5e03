"""Residual addition and root-mean-square norm (include/q4k_layer.h) against 64 bits."""
import numpy as np
import pytest

import gguf_q4_dequant_amd as q4k
from tests.gpu_helpers import to_dev
from tests.layer_reference import rng_of

pytestmark = pytest.mark.gpu

# total is one float32 addition.  y: total, its factor, their product and the
# product with the weight are each rounded once (2^-24), the factor from a double.
Y_TOL = 5 * 2.0 ** -24


def plain(x, residual, weight, eps):
    t = x.astype(np.float64) + (0 if residual is None else residual.astype(np.float64))
    return t / np.sqrt((t * t).mean(1, keepdims=True) + eps) * weight.astype(np.float64)


SIZES = [(1, 1), (1, 3), (3, 4), (2, 255), (1, 2048), (5, 1023), (4, 1025), (7, 4096), (1, 4097), (3, 5120), (2, 16384),
         (1, 16387), (2, 40001), (300, 640), (2049, 130)]


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("M,N", SIZES)
def test_norm(M, N, residual):
    rng = rng_of(1, M, N, int(residual))
    x = rng.standard_normal((M, N)).astype(np.float32) * np.where(rng.random((1, N)) < 0.02, 30, 1).astype(np.float32)
    r = rng.standard_normal((M, N)).astype(np.float32) if residual else None
    w = (rng.random(N) * 2 - 0.5).astype(np.float32)
    got = q4k.rms_norm(to_dev(x), to_dev(w), 1e-5, residual=None if r is None else to_dev(r))
    if residual:
        got, total = got
        assert np.array_equal(total.cpu().numpy(), x + r)
    want = plain(x, r, w, 1e-5)
    # where the sum cancels its rounding (2^-24 of the addends) counts beside the value
    slack = 0 if r is None else 2.0 ** -24 * (np.abs(want) + np.abs(w) * (np.abs(x) + np.abs(r)) /
                                              np.sqrt(((x + r).astype(np.float64) ** 2).mean(1, keepdims=True)))
    assert (np.abs(got.cpu().numpy() - want) <= Y_TOL * np.abs(want) + slack).all()


def test_in_place_and_given_outputs():
    import torch
    rng = rng_of(2)
    x, r, w = (rng.standard_normal(s).astype(np.float32) for s in ((6, 777), (6, 777), (777,)))
    y, t = q4k.rms_norm(to_dev(x), to_dev(w), residual=to_dev(r))
    xd, rd, wd = to_dev(x), to_dev(r), to_dev(w)
    y2, t2 = q4k.rms_norm(xd, wd, residual=rd, total=rd, out=xd)
    assert y2 is xd and t2 is rd and torch.equal(y, xd) and torch.equal(t, rd)
    xd, rd = to_dev(x), to_dev(r)
    y3, t3 = q4k.rms_norm(xd, wd, residual=rd, total=xd, out=rd)
    assert torch.equal(y, rd) and torch.equal(t, xd)
    xd, extra = to_dev(x), torch.empty(6, 777, device="cuda")
    y4 = q4k.rms_norm(xd, wd, total=extra, out=xd)
    assert y4 is xd and np.array_equal(extra.cpu().numpy(), x)


def test_unusual_rows():
    x = np.ones((6, 300), np.float32)
    x[0] = 0
    x[1, 5] = np.nan
    x[2, 7] = np.inf
    x[3] = 1e30   # squares past float32's range
    x[4] = 1e-30
    w = np.full(300, 2, np.float32)
    y = q4k.rms_norm(to_dev(x), to_dev(w), 0.0).cpu().numpy()
    assert np.isnan(y[0]).all()  # 0 * rsqrt(0), as the formula says
    assert np.isnan(y[1]).all()
    assert np.isnan(y[2, 7]) and (np.delete(y[2], 7) == 0).all()
    assert np.allclose(y[3:6], 2, rtol=1e-6)
    y = q4k.rms_norm(to_dev(x[:1]), to_dev(w), 1e-6).cpu().numpy()
    assert (y == 0).all()


def test_rows_at_odd_addresses():
    import torch
    base = torch.randn(5 * 301 + 1, device="cuda")
    x = base[1:].view(5, 301)  # 4-byte aligned only
    w = torch.rand(302, device="cuda")[1:]
    want = plain(x.cpu().numpy(), None, w.cpu().numpy(), 1e-6)
    got = q4k.rms_norm(x, w).cpu().numpy()
    assert (np.abs(got - want) <= Y_TOL * np.abs(want)).all()


def test_empty():
    import torch
    assert q4k.rms_norm(torch.zeros(0, 8, device="cuda"), torch.zeros(8, device="cuda")).shape == (0, 8)
    assert q4k.rms_norm(torch.zeros(3, 0, device="cuda"), torch.zeros(0, device="cuda")).shape == (3, 0)


def test_refusals():
    import torch
    x, w = torch.zeros(3, 8, device="cuda"), torch.zeros(8, device="cuda")
    with pytest.raises(ValueError, match="weight"):
        q4k.rms_norm(x, w[:7])
    with pytest.raises(ValueError, match="residual"):
        q4k.rms_norm(x, w, residual=x[:2])
    with pytest.raises(ValueError, match="contiguous"):
        q4k.rms_norm(x.t(), x.new_zeros(3))
    with pytest.raises(ValueError, match="two tensors"):
        o = torch.empty_like(x)
        q4k.rms_norm(x, w, residual=x, total=o, out=o)
