"""hipStreamPerThread is one handle for a stream of every thread: each thread's calls on it have a
workspace of their own."""
import threading

import numpy as np
import pytest

import gguf_q4_dequant_amd as q4k
import q4k_inputs as qi
from tests.gpu_helpers import to_dev
from tests.layer_reference import Paged, rng_of

pytestmark = pytest.mark.gpu

LEGACY, PER_THREAD = 1, 2  # hipStreamLegacy, hipStreamPerThread


def in_threads(work, repeats):
    """work: (call, out, want) of each thread; every call of every thread gives its own result."""
    import torch
    bad = []
    start = threading.Barrier(len(work))

    def run(call, out, want):
        start.wait()
        for _ in range(repeats):
            out.fill_(float("nan"))
            torch.cuda.current_stream().synchronize()  # (the fill is the default stream's)
            call()
            torch.cuda.ExternalStream(PER_THREAD).synchronize()
            if not torch.equal(out, want):
                bad.append(1)

    threads = [threading.Thread(target=run, args=w) for w in work]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert not bad


def test_attention():
    import torch
    work = []
    for n in range(4):
        rng = rng_of(110, n)
        p = Paged(rng, [(2000 + 100 * n, 1 + 8 * (n % 2)), (50, 1)], 2, 64, 16, "f16")
        cache, seqs = p.on_device()
        q = to_dev(rng.standard_normal((p.T, 8, 64)).astype(np.float32))
        want, out = q4k.attention(q, cache, seqs), torch.empty_like(q)
        work.append((lambda q=q, c=cache, s=seqs, o=out: q4k.attention(q, c, s, out=o, stream=PER_THREAD), out, want))
    torch.cuda.synchronize()
    in_threads(work, 30)


def test_products():
    """Ten tokens: the activations are staged in the workspace."""
    import torch
    work = []
    for n in range(4):
        K, N = 2048 + 256 * n, 500
        w = to_dev(qi.random_q4k(N, K, seed=qi.tensor_seed(qi.BASE_SEED, 1110, n)))
        x = to_dev(qi.random_x(10, K, seed=qi.tensor_seed(qi.BASE_SEED, 1111, n)))
        y = torch.empty(10, N, device="cuda")
        want = q4k.matmul(w, x)
        work.append((lambda w=w, x=x, y=y: q4k.matmul(w, x, y, stream=PER_THREAD), y, want))
    torch.cuda.synchronize()
    in_threads(work, 30)


def test_beside_the_null_streams_own_handle():
    """One thread's calls on its stream, another's on hipStreamLegacy: two workspaces.  (The legacy stream
    waits for blocking streams, and the per-thread stream is one, so they do not run at once here; the
    results say that neither call takes the other's counters or parts.)"""
    import torch
    work = []
    for n, handle in enumerate((PER_THREAD, LEGACY)):
        rng = rng_of(111, n)
        p = Paged(rng, [(2500 - 700 * n, 1), (50, 1)], 2, 64, 16, "f16")
        cache, seqs = p.on_device()
        q = to_dev(rng.standard_normal((p.T, 8, 64)).astype(np.float32))
        want, out = q4k.attention(q, cache, seqs), torch.empty_like(q)
        work.append((lambda q=q, c=cache, s=seqs, o=out, h=handle: (q4k.attention(q, c, s, out=o, stream=h),
                                                                    torch.cuda.synchronize()), out, want))
    torch.cuda.synchronize()
    in_threads(work, 20)
