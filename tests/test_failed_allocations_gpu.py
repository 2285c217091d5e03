"""A call that could not allocate its workspace leaves nothing behind that a later call reports."""
import ctypes

import numpy as np
import pytest

import gguf_q4_dequant_amd as q4k
import q4k_inputs as qi
from tests.gpu_helpers import fresh_stream, to_dev
from tests.layer_reference import Paged, rng_of

pytestmark = pytest.mark.gpu


def _attention():
    rng = rng_of(120)
    p = Paged(rng, [(900, 1), (40, 1)], 2, 64, 16, "f16")
    cache, seqs = p.on_device()
    q = to_dev(rng.standard_normal((2, 8, 64)).astype(np.float32))
    out = q.clone()
    return lambda st: q4k.attention(q, cache, seqs, out=out, stream=st)


def _matmul():
    import torch
    w = to_dev(qi.random_q4k(300, 2048, seed=qi.tensor_seed(qi.BASE_SEED, 1120, 0)))
    x = to_dev(qi.random_x(64, 2048, seed=qi.tensor_seed(qi.BASE_SEED, 1120, 1)))
    y = torch.empty(64, 300, device="cuda")
    return lambda st: q4k.matmul(w, x, y, stream=st)


@pytest.mark.parametrize("make", [_attention, _matmul])
def test_the_next_call_succeeds(make):
    """Inside a global capture nothing can be allocated: the call is refused (and the capture is lost), and
    the next one, on a stream that has its workspace, is not."""
    import torch
    hip = ctypes.CDLL("libamdhip64.so")
    call = make()
    want = call(None).clone()
    x, w, y = torch.randn(3, 64, device="cuda"), torch.rand(64, device="cuda"), torch.empty(3, 64, device="cuda")
    side, other = fresh_stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    assert hip.hipStreamBeginCapture(ctypes.c_void_p(side.cuda_stream), 0) == 0
    try:
        with pytest.raises(q4k.Q4KError):
            call(side)
        q4k.rms_norm(x, w, out=y, stream=other)
    finally:
        graph = ctypes.c_void_p()
        hip.hipStreamEndCapture(ctypes.c_void_p(side.cuda_stream), ctypes.byref(graph))
        hip.hipGetLastError()
    torch.cuda.synchronize()
    assert torch.equal(y, q4k.rms_norm(x, w))
    assert torch.equal(call(other), want)  # (side is of no more use: HIP keeps its capture's error)
    torch.cuda.synchronize()
