"""Outputs that the binding makes for a call on a given stream come from that
stream's memory: on the current stream's, a tensor freed there a moment ago,
whose last kernels have not run, would be written over."""
import numpy as np
import pytest

import gguf_q4_dequant_amd as q4k
import q4k_inputs as qi
from tests.gpu_helpers import to_dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def side():
    """One stream for all (torch hands out the same 32 in turn)."""
    import torch
    return torch.cuda.Stream()


def _memory_stream(t):
    import torch
    at = t.data_ptr()
    for segment in torch.cuda.memory_snapshot():
        if segment["address"] <= at < segment["address"] + segment["total_size"]:
            return segment["stream"]
    raise AssertionError("not in the allocator's memory")


def _calls():
    import torch
    E, M, k, K, N = 4, 3, 2, 512, 96
    w = to_dev(np.stack([qi.random_q4k(N, K, seed=e) for e in range(E)]))
    x, xp = to_dev(qi.random_x(M, K, seed=1)), to_dev(qi.random_x(M * k, K, seed=2))
    logits = to_dev(qi.random_x(M, E, seed=3))
    r = q4k.moe_route(logits, k)
    a = q4k.Adjustment(history=torch.zeros((M, 2), dtype=torch.int32, device="cuda"))
    z = to_dev(qi.random_x(M, 300, seed=4))
    aq, s, b = (to_dev(v) for v in qi.random_q4a(N, K, seed=5))
    return {
        "moe_route": lambda st: q4k.moe_route(logits, k, stream=st),
        "moe_group": lambda st: q4k.moe_group(r.expert, E, stream=st),
        "matmul_grouped": lambda st: q4k.matmul_grouped(w, x, r.offsets, r.rows, x_div=k, stream=st),
        "matmul_grouped_swiglu": lambda st: q4k.matmul_grouped_swiglu(w, w, x, r.offsets, r.rows, x_div=k, stream=st),
        "matmul_grouped_combine": lambda st: q4k.matmul_grouped_combine(w, xp, r, stream=st),
        "logits_adjust": lambda st: q4k.logits_adjust(z, a, stream=st),
        "logits_argmax": lambda st: q4k.logits_argmax(z, a, stream=st),
        "matmul_argmax": lambda st: q4k.matmul_argmax(w[0], x, stream=st),
        "matmul_argmax adjusted": lambda st: q4k.matmul_argmax(w[0], x, adjustment=a, stream=st),
        "matmul": lambda st: q4k.matmul(w[0], x, stream=st),
        "matmul_swiglu": lambda st: q4k.matmul_swiglu(w[0], w[1], x, stream=st),
        "q4a_matmul": lambda st: q4k.q4a_matmul(aq, s, b, x, stream=st),
    }


CALLS = ["moe_route", "moe_group", "matmul_grouped", "matmul_grouped_swiglu", "matmul_grouped_combine", "logits_adjust",
         "logits_argmax", "matmul_argmax", "matmul_argmax adjusted", "matmul", "matmul_swiglu", "q4a_matmul"]


@pytest.mark.parametrize("handle", [False, True], ids=["stream", "handle"])
@pytest.mark.parametrize("call", CALLS)
def test_outputs_come_from_the_given_streams_memory(call, handle, side):
    import torch
    run = _calls()[call]
    want = run(None)
    torch.cuda.synchronize()
    got = run(side.cuda_stream if handle else side)
    assert torch.cuda.current_stream() == torch.cuda.default_stream()
    torch.cuda.synchronize()
    want, got = [t if isinstance(t, tuple) else (t,) for t in (want, got)]
    for a, b in zip(want, got):
        assert _memory_stream(a) == 0 and _memory_stream(b) == side.cuda_stream
        assert torch.equal(a, b)


def test_the_default_stream_by_its_handle(side):
    import torch
    run = _calls()["matmul_grouped"]
    with torch.cuda.stream(side):
        side.wait_stream(torch.cuda.default_stream())
        y = run(0)
    torch.cuda.synchronize()
    assert _memory_stream(y) == 0 and torch.equal(y, run(None))
