"""Penalties, biases and grammar masks on logits, and the greedy choice under
them (include/q4k_select.h).  The definition is a fixed sequence of float32
operations, so the adjusted logits are compared bit for bit with numpy's."""
import numpy as np
import pytest

import gguf_q4_dequant_amd as q4k
import q4k_inputs as qi
from tests.gpu_helpers import device, to_dev

pytestmark = pytest.mark.gpu


def _rng(*path):
    return np.random.Generator(np.random.PCG64(qi.tensor_seed(qi.BASE_SEED, 1200, *path)))


def plain(z, history=None, repetition=None, frequency=None, presence=None, bias_id=None, bias_value=None, mask=None):
    """The definition, one token at a time, in float32."""
    f = np.float32
    z = z.copy()
    M, N = z.shape
    with np.errstate(all="ignore"):
        for m in range(M):
            if history is not None:
                ids = history[m]
                for n, c in zip(*np.unique(ids[(ids >= 0) & (ids < N)], return_counts=True)):
                    r = f(1) if repetition is None else repetition[m]
                    q = f(0) if frequency is None else frequency[m]
                    p = f(0) if presence is None else presence[m]
                    t = f(z[m, n] / r) if z[m, n] > 0 else f(z[m, n] * r)
                    z[m, n] = f(f(t - f(q * f(c))) - p)
            if bias_id is not None:
                sums = {}
                for n, b in zip(bias_id[m], bias_value[m]):
                    if 0 <= n < N:
                        sums[n] = f(sums.get(n, f(0)) + b)
                for n, b in sums.items():
                    z[m, n] = f(z[m, n] + b)
            if mask is not None:
                bits = (mask[m].view(np.uint32)[:, None] >> np.arange(32, dtype=np.uint32)) & 1
                z[m, bits.reshape(-1)[:N] == 0] = -np.inf
    return z


def choice(z, mask):
    """(index, value): the first largest among allowed tokens that are not NaN."""
    M, N = z.shape
    index, value = np.full(M, -1, np.int32), np.full(M, -np.inf, np.float32)
    for m in range(M):
        ok = ~np.isnan(z[m])
        if mask is not None:
            bits = (mask[m].view(np.uint32)[:, None] >> np.arange(32, dtype=np.uint32)) & 1
            ok &= bits.reshape(-1)[:N] == 1
        if ok.any():
            v = np.where(ok, z[m], -np.inf)
            best = v.max()
            index[m] = np.argmax(ok & (v == best))
            value[m] = best
    return index, value


def _case(M, N, L, B, masked, tag=0):
    g = _rng(M, N, L, B, tag)
    z = (4 * g.standard_normal((M, N))).astype(np.float32)
    c = {}
    if L:
        c["history"] = g.integers(-2, N + 3, (M, L)).astype(np.int32)  # padding and ids past the end
        c["history"][:, ::3] = c["history"][:, :1]                     # one token again and again
        c["repetition"] = (1 + g.random(M)).astype(np.float32)
        c["frequency"] = g.random(M).astype(np.float32)
        c["presence"] = g.standard_normal(M).astype(np.float32)
    if B:
        c["bias_id"] = g.integers(-2, N + 3, (M, B)).astype(np.int32)
        c["bias_id"][:, B // 2] = c["bias_id"][:, 0]                   # the same token twice
        c["bias_value"] = (5 * g.standard_normal((M, B))).astype(np.float32)
    if masked:
        c["mask"] = g.integers(-2 ** 31, 2 ** 31, (M, (N + 31) // 32)).astype(np.int32)
    return z, c


def _adjustment(c):
    return q4k.Adjustment(**{n: to_dev(v) for n, v in c.items()})


def _check(z, c):
    import torch
    a, zd = _adjustment(c), to_dev(z)
    want = plain(z, **c)
    out = q4k.logits_adjust(zd, a)
    index, value = q4k.logits_argmax(zd, a)
    torch.cuda.synchronize()
    assert np.array_equal(out.cpu().numpy(), want, equal_nan=True)
    wi, wv = choice(want, c.get("mask"))
    assert np.array_equal(index.cpu().numpy(), wi)
    assert np.array_equal(value.cpu().numpy(), wv)
    assert np.array_equal(zd.cpu().numpy(), z, equal_nan=True)  # the logits are only read
    q4k.logits_adjust(zd, a, out=zd)                            # in place
    assert np.array_equal(zd.cpu().numpy(), want, equal_nan=True)


@pytest.mark.parametrize("L,B,masked", [(0, 0, True), (1, 0, False), (0, 1, False), (40, 3, True), (700, 33, True)])
@pytest.mark.parametrize("M,N", [(1, 1), (2, 31), (3, 33), (1, 1023), (2, 1025), (5, 4097), (1, 50257)])
def test_adjusted_logits_and_choice(M, N, L, B, masked):
    _check(*_case(M, N, L, B, masked))


@pytest.mark.parametrize("M,N,L,B,masked", [(40, 32001, 300, 9, True), (9, 151936, 65, 0, False), (300, 4096, 0, 4, True)])
def test_many_logits(M, N, L, B, masked):
    """More than 2^20 logits in a call: the larger chunks."""
    _check(*_case(M, N, L, B, masked))


def test_parts_of_the_penalties_may_be_left_out():
    z, c = _case(3, 777, 20, 0, False)
    for leave in ("repetition", "frequency", "presence"):
        _check(z, {n: v for n, v in c.items() if n != leave})
    _check(z, {"history": c["history"]})
    _check(z, {})


@pytest.mark.parametrize("N", [50, 3000])
def test_masks_that_leave_nothing_and_unusual_logits(N):
    z, c = _case(8, N, 10, 2, True)
    c["mask"][0] = 0                                  # nothing allowed
    c["mask"][1] = 0
    c["mask"][1, (N - 1) // 32] = np.uint32(1 << ((N - 1) % 32)).astype(np.int32)  # only the last token
    z[2] = np.nan                                     # nothing but NaN
    z[3, ::2] = np.nan
    z[4] = -np.inf                                    # allowed, but -inf
    z[5, N // 2] = np.inf
    z[6] = np.finfo(np.float32).min
    bits = (c["mask"][7].view(np.uint32)[:, None] >> np.arange(32, dtype=np.uint32)) & 1
    z[7, bits.reshape(-1)[:N] == 0] = np.nan          # NaN in masked places only
    _check(z, c)
    assert np.isfinite(plain(z, **c)[7][bits.reshape(-1)[:N] == 1]).all()


def test_equal_logits_give_the_lowest_allowed_token():
    z = np.zeros((4, 9000), np.float32)
    mask = np.full((4, (9000 + 31) // 32), -1, np.int32)
    mask[1, :100] = 0
    mask[2, 0] = ~1
    mask[3, :] = 0
    mask[3, 200] = -2 ** 31
    index, value = q4k.logits_argmax(to_dev(z), q4k.Adjustment(mask=to_dev(mask)))
    assert index.tolist() == [0, 3200, 1, 6431] and value.tolist() == [0.0] * 4


@pytest.mark.parametrize("M,N,K", [(1, 5000, 1024), (3, 4097, 512), (20, 3000, 512)])
def test_head_under_an_adjustment(M, N, K):
    """matmul_argmax with an Adjustment = the library's own product, adjusted."""
    import torch
    w, x = to_dev(qi.random_q4k(N, K, seed=7)), to_dev(qi.random_x(M, K, seed=8))
    _, c = _case(M, N, 30, 4, True)
    a = _adjustment(c)
    index, value = q4k.matmul_argmax(w, x, adjustment=a)
    logits = q4k.matmul(w, x)
    torch.cuda.synchronize()
    wi, wv = choice(plain(logits.cpu().numpy(), **c), c["mask"])
    assert np.array_equal(index.cpu().numpy(), wi) and np.array_equal(value.cpu().numpy(), wv)


def test_greedy_steps_captured_and_replayed():
    """A step of constrained greedy decoding (head, penalties, mask, choice),
    captured once; the history grows between the replays."""
    import torch
    M, N, K, L = 2, 6000, 512, 16
    w = to_dev(qi.random_q4k(N, K, seed=17))
    x = to_dev(qi.random_x(M, K, seed=18))
    _, c = _case(M, N, L, 2, True)
    c["history"][:] = -1
    a = _adjustment(c)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        q4k.matmul_argmax(w, x, adjustment=a)  # grows the workspace before the capture
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        index, value = q4k.matmul_argmax(w, x, adjustment=a)
    seen = []
    for step in range(4):
        graph.replay()
        torch.cuda.synchronize()
        got = index.clone(), value.clone()
        eager = q4k.matmul_argmax(w, x, adjustment=a)
        torch.cuda.synchronize()
        assert torch.equal(got[0], eager[0]) and torch.equal(got[1], eager[1]), step
        a.history[:, step] = got[0]
        seen.append(got[1].tolist())
    logits = q4k.matmul(w, x).cpu().numpy()
    c["history"] = a.history.cpu().numpy()
    wi, wv = choice(plain(logits, **c), c["mask"])
    assert np.array_equal(q4k.matmul_argmax(w, x, adjustment=a)[0].cpu().numpy(), wi)


def test_no_rows():
    import torch
    z = torch.empty((0, 40), device=device())
    mask = torch.empty((0, 2), dtype=torch.int32, device=device())
    assert q4k.logits_adjust(z, q4k.Adjustment(mask=mask)).shape == (0, 40)
    index, value = q4k.logits_argmax(z, q4k.Adjustment(mask=mask))
    assert index.shape == (0,) and value.shape == (0,)
