"""Mixture-of-experts operators (include/q4k_moe.h) against plain 64-bit forms:
routing and grouping, grouped products, their SwiGLU form, the weighted sum,
and a whole layer of them."""
import numpy as np
import pytest

import gguf_q4_dequant_amd as q4k
import q4k_inputs as qi
from tests import moe_reference as ref
from tests.gpu_helpers import check_close, device, to_dev

pytestmark = pytest.mark.gpu


def _rng(*path):
    return np.random.Generator(np.random.PCG64(qi.tensor_seed(qi.BASE_SEED, 1100, *path)))


# ---- routing -----------------------------------------------------------------

def _check_route(logits, top_k, bias=None, sigmoid=False, normalize=True, scale=1.0):
    E = logits.shape[1]
    r = q4k.moe_route(to_dev(logits), top_k, bias=None if bias is None else to_dev(bias), sigmoid=sigmoid,
                      normalize=normalize, scale=scale)
    expert, weight = ref.route(logits, bias, top_k, sigmoid, normalize, scale)
    got = r.expert.cpu().numpy()
    assert np.array_equal(got, expert)
    # exp of a difference d is off by |d| * 2^-24 and a few ulp; sums of up to E
    # terms, a quotient and two products add theirs
    finite = logits[np.isfinite(logits)]
    spread = float(finite.max() - finite.min()) if finite.size else 0.0
    tol = (spread + 16 + np.sqrt(E)) * 2.0 ** -23
    w = r.weight.cpu().numpy().astype(np.float64)
    assert np.all(np.abs(w - weight) <= tol * np.abs(weight) + 1e-37), np.abs(w - weight).max()
    offsets, rows = ref.stable_groups(expert, E)
    assert np.array_equal(r.offsets.cpu().numpy(), offsets)
    assert np.array_equal(r.rows.cpu().numpy(), rows)


@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("sigmoid,normalize", [(False, True), (False, False), (True, True), (True, False)])
@pytest.mark.parametrize("M,E,k", [(1, 1, 1), (1, 128, 8), (3, 7, 7), (64, 65, 3), (65, 64, 64), (130, 257, 16),
                                   (1025, 1024, 5), (2500, 96, 2)])
def test_route(M, E, k, sigmoid, normalize, bias):
    g = _rng(1, M, E, k)
    logits = (2.0 * g.standard_normal((M, E))).astype(np.float32)
    b = (0.2 * g.standard_normal(E)).astype(np.float32) if bias else None
    _check_route(logits, k, b, sigmoid, normalize, scale=1.0 if normalize else 2.5)


@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("M,E,k", [(16, 300, 64), (17, 300, 2), (48, 513, 7), (49, 513, 7), (2, 1024, 64), (16, 1024, 1)])
def test_route_around_the_change_of_kernels(M, E, k, bias):
    g = _rng(8, M, E, k)
    logits = (2.0 * g.standard_normal((M, E))).astype(np.float32)
    _check_route(logits, k, (0.2 * g.standard_normal(E)).astype(np.float32) if bias else None, sigmoid=bias)
    # few different scores: every choice is among equals
    _check_route(np.round(logits), k, np.zeros(E, np.float32) if bias else None, sigmoid=not bias)


@pytest.mark.parametrize("M", [5, 200])
@pytest.mark.parametrize("bias", [False, True])
def test_route_equal_scores_go_to_the_lower_expert(M, bias):
    g = _rng(2, M)
    logits = g.integers(-2, 3, (M, 150)).astype(np.float32)  # many ties
    b = np.zeros(150, np.float32) if bias else None
    _check_route(logits, 9, b, sigmoid=True)
    _check_route(np.zeros((M, 150), np.float32), 20, b)


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("bias", [False, True])
def test_route_masked_nan_and_infinite_logits(sigmoid, bias):
    g = _rng(3)
    logits = g.standard_normal((70, 40)).astype(np.float32)
    logits[0] = -np.inf                      # nothing left
    logits[1] = np.nan
    logits[2, 3:] = -np.inf                  # three left, six wanted
    logits[3, ::2] = np.nan
    logits[4, 7] = np.inf
    logits[5, [1, 30]] = np.inf
    logits[6] = np.finfo(np.float32).min     # a mask's lowest value: all equal
    logits[7, :] = -200.0                    # sigmoid underflows
    logits[8, 5] = np.finfo(np.float32).max
    b = (0.1 * g.standard_normal(40)).astype(np.float32) if bias else None
    if bias:
        b[11] = -np.inf                      # never chosen
        b[12] = np.nan
    E = 40
    r = q4k.moe_route(to_dev(logits), 6, bias=None if b is None else to_dev(b), sigmoid=sigmoid)
    expert, weight = ref.route(logits, b, 6, sigmoid, True, 1.0)
    assert np.array_equal(r.expert.cpu().numpy(), expert)
    w = r.weight.cpu().numpy().astype(np.float64)
    # as above with differences up to 200; float32 underflow leaves up to 2^-126
    assert np.all(np.abs(w - weight) <= 256 * 2.0 ** -23 * weight + 2.0 ** -126)
    offsets, rows = ref.stable_groups(expert, E)
    assert np.array_equal(r.offsets.cpu().numpy(), offsets) and np.array_equal(r.rows.cpu().numpy(), rows)


def test_route_of_no_tokens_writes_empty_groups():
    import torch
    r = q4k.moe_route(torch.empty((0, 9), device=device()), 2)
    assert r.offsets.tolist() == [0] * 10 and r.rows.numel() == 0


@pytest.mark.parametrize("P", [0, 1, 63, 64, 65, 1000, 8192, 8193, 100000])
@pytest.mark.parametrize("E", [1, 3, 64, 1000])
def test_group(P, E):
    expert = _rng(4, P, E).integers(-1, E + 1, P).astype(np.int32)  # -1 and E: no group
    offsets, rows = q4k.moe_group(to_dev(expert), E)
    want_offsets, want_rows = ref.stable_groups(expert, E)
    assert np.array_equal(offsets.cpu().numpy(), want_offsets)
    assert np.array_equal(rows.cpu().numpy(), want_rows)


# ---- grouped products -----------------------------------------------------------

def _weights(E, N, K, tag):
    return np.stack([qi.random_q4k(N, K, seed=qi.tensor_seed(qi.BASE_SEED, 1101, tag, e, N, K)) for e in range(E)])


def _table(sizes, tag):
    """offsets and shuffled rows for groups of these sizes."""
    P = int(sum(sizes))
    rows = _rng(5, tag, P).permutation(P).astype(np.int32)
    offsets = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    for e in range(len(sizes)):
        rows[offsets[e]:offsets[e + 1]].sort()
    return offsets, rows, P


SIZES = [
    [1], [0, 1], [1] * 8 + [0] * 8, [3, 0, 17, 16, 15, 1], [64, 63, 65, 0, 129], [300, 2, 0, 40], [5, 7, 0, 0, 33, 9],
    [0, 0, 700], [31, 32, 33, 34], [0] * 30 + [9, 4], [2, 5, 0, 0, 1, 0, 0, 3],
]


@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: "-".join(map(str, s[:6])))
@pytest.mark.parametrize("N,K,x_div", [(1, 256, 1), (33, 512, 2), (300, 1024, 8), (129, 2304, 1)])
def test_grouped_product(sizes, N, K, x_div):
    import torch
    offsets, rows, P = _table(sizes, N)
    w = _weights(len(sizes), N, K, 1)
    x = qi.random_x((P + x_div - 1) // x_div, K, seed=qi.tensor_seed(qi.BASE_SEED, 1102, P, K))
    y = q4k.matmul_grouped(to_dev(w), to_dev(x), to_dev(offsets), to_dev(rows), x_div=x_div)
    torch.cuda.synchronize()
    want, s = ref.grouped(w, x, offsets, rows, x_div, P)
    check_close(y.cpu().numpy(), want, s, ref.product_tol(K))


@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: "-".join(map(str, s[:6])))
@pytest.mark.parametrize("N,K,x_div", [(1, 256, 1), (47, 512, 2), (200, 1280, 8)])
def test_grouped_swiglu(sizes, N, K, x_div):
    import torch
    offsets, rows, P = _table(sizes, N)
    wg, wu = _weights(len(sizes), N, K, 2), _weights(len(sizes), N, K, 3)
    x = (0.02 * qi.random_x((P + x_div - 1) // x_div, K, seed=qi.tensor_seed(qi.BASE_SEED, 1103, P, K))).astype(np.float32)
    out = q4k.matmul_grouped_swiglu(to_dev(wg), to_dev(wu), to_dev(x), to_dev(offsets), to_dev(rows), x_div=x_div)
    torch.cuda.synchronize()
    g, sg = ref.grouped(wg, x, offsets, rows, x_div, P)
    u, su = ref.grouped(wu, x, offsets, rows, x_div, P)
    want = ref.silu(g) * u
    # |silu'| < 1.1; the exponential's argument carries |g| * 2^-23, the rest a few ulp
    t = ref.product_tol(K)
    bound = 1.1 * t * sg * (np.abs(u) + t * su) + np.abs(ref.silu(g)) * t * su + np.abs(want) * (np.abs(g) + 8) * 2.0 ** -23
    err = np.abs(out.cpu().numpy().astype(np.float64) - want)
    assert np.all(err <= bound + 1e-30), (err / (bound + 1e-30)).max()


# One call of each kernel that the sizes choose: four-row tiles on four and
# eight waves, sixteen-row tiles with K over four, two and one groups of waves,
# 32 x 128 and 48 x 256 tiles.  The groups' sizes are uneven and some are empty.
@pytest.mark.parametrize("P,E,N,K", [(40, 2, 300, 512), (40, 2, 300, 1280), (200, 2, 1000, 1024), (400, 2, 1000, 512),
                                     (200, 24, 2600, 512), (3000, 2, 300, 512), (3000, 2, 2300, 256),
                                     (900, 600, 40, 256), (5000, 300, 150, 256), (70, 1024, 33, 512),
                                     (3000, 2, 5000, 256), (5000, 3, 2600, 512)])
def test_every_kernel(P, E, N, K):
    import torch
    g = _rng(7, P, E)
    share = g.random(E) ** 2
    share[::7] = 0.0 if E > 2 else share[::7]
    offsets, rows, P = _table(g.multinomial(P, share / share.sum()), P)
    w, u = _weights(E, N, K, 20), _weights(E, N, K, 21)
    x = (0.02 * qi.random_x((P + 1) // 2, K, seed=P)).astype(np.float32)
    args = to_dev(x), to_dev(offsets), to_dev(rows)
    y = q4k.matmul_grouped(to_dev(w), *args, x_div=2)
    h = q4k.matmul_grouped_swiglu(to_dev(w), to_dev(u), *args, x_div=2)
    torch.cuda.synchronize()
    want, s = ref.grouped(w, x, offsets, rows, 2, P)
    check_close(y.cpu().numpy(), want, s, ref.product_tol(K))
    wu, su = ref.grouped(u, x, offsets, rows, 2, P)
    t = ref.product_tol(K)  # as in test_grouped_swiglu
    bound = 1.1 * t * s * (np.abs(wu) + t * su) + np.abs(ref.silu(want)) * t * su + \
        np.abs(ref.silu(want) * wu) * (np.abs(want) + 8) * 2.0 ** -23
    err = np.abs(h.cpu().numpy().astype(np.float64) - ref.silu(want) * wu)
    assert np.all(err <= bound + 1e-30), (err / (bound + 1e-30)).max()


@pytest.mark.parametrize("M,E,k,N,K", [(1, 8, 2, 96, 512), (3, 4, 4, 33, 256), (40, 16, 3, 260, 768), (257, 5, 2, 64, 512),
                                       (1, 64, 8, 300, 1280)])
@pytest.mark.parametrize("holes", [False, True])
def test_grouped_combine(M, E, k, N, K, holes):
    import torch
    g = _rng(6, M, E, k)
    expert = np.argsort(g.random((M, E)), axis=1)[:, :k].astype(np.int32)
    if holes:  # padded tokens and unused choices
        expert[g.random((M, k)) < 0.4] = -1
        expert[M // 2] = -1
    weight = g.random((M, k)).astype(np.float32)
    offsets, rows = ref.stable_groups(expert, E)
    w = _weights(E, N, K, 4)
    x = qi.random_x(M * k, K, seed=qi.tensor_seed(qi.BASE_SEED, 1104, M, K))
    r = q4k.Routing(to_dev(expert), to_dev(weight), to_dev(offsets), to_dev(rows))
    out = q4k.matmul_grouped_combine(to_dev(w), to_dev(x), r)
    torch.cuda.synchronize()
    y, s = ref.grouped(w, x, offsets, rows[:offsets[-1]], 1, M * k)
    y, s = np.nan_to_num(y).reshape(M, k, N), np.nan_to_num(s).reshape(M, k, N)
    want = (weight[:, :, None].astype(np.float64) * y).sum(1)
    # the products' error, and k fused multiply-adds of at most 2^-24 of sum |weight| |y| each
    bound = (weight[:, :, None] * s).sum(1) * (ref.product_tol(K) + k * 2.0 ** -24)
    err = np.abs(out.cpu().numpy().astype(np.float64) - want)
    assert np.all(err <= bound), (err / np.maximum(bound, 1e-30)).max()
    if holes:
        assert np.all(out.cpu().numpy()[M // 2] == 0.0)


def test_rows_of_no_group_are_left_as_they_were_and_bad_entries_skipped():
    import torch
    E, N, K, P = 4, 70, 512, 50
    w = _weights(E, N, K, 5)
    x = qi.random_x(P, K, seed=5)
    rows = np.arange(P, dtype=np.int32)
    rows[3], rows[20], rows[21] = -1, P, np.iinfo(np.int32).max  # outside [0, P): skipped
    offsets = np.array([0, 10, 10, 25, 30], np.int32)            # 30 .. 49 in no group
    y = torch.full((P, N), 7.0, device=device())
    q4k.matmul_grouped(to_dev(w), to_dev(x), to_dev(offsets), to_dev(rows), y=y)
    torch.cuda.synchronize()
    want, s = ref.grouped(w, x, offsets, rows, 1, P)
    got = y.cpu().numpy()
    left = np.isnan(want[:, 0])
    assert left.sum() == 23
    assert np.all(got[left] == 7.0)
    check_close(got[~left], want[~left], s[~left], ref.product_tol(K))
    # offsets behind the table's end and descending ones: clamped, an empty group
    bad = np.array([0, 10, 4, 60, 70], np.int32)
    y.fill_(7.0)
    q4k.matmul_grouped(to_dev(w), to_dev(x), to_dev(bad), to_dev(rows), y=y)
    torch.cuda.synchronize()
    assert np.all(y.cpu().numpy()[[3, 20, 21]] == 7.0)


def test_rows_may_be_left_out_when_pairs_come_in_expert_order():
    sizes = [4, 0, 19, 2]
    offsets, _, P = _table(sizes, 9)
    w, x = _weights(4, 65, 768, 6), qi.random_x(P, 768, seed=9)
    y = q4k.matmul_grouped(to_dev(w), to_dev(x), to_dev(offsets))
    want, s = ref.grouped(w, x, offsets, np.arange(P), 1, P)
    check_close(y.cpu().numpy(), want, s, ref.product_tol(768))


def test_empty_calls_do_nothing():
    import torch
    dev = device()
    w, x = to_dev(_weights(3, 20, 256, 16)), torch.empty((0, 256), device=dev)
    r = q4k.moe_route(torch.empty((0, 3), device=dev), 2)
    assert q4k.matmul_grouped(w, x, r.offsets, r.rows).shape == (0, 20)
    assert q4k.matmul_grouped_swiglu(w, w, x, r.offsets, r.rows, x_div=2).shape == (0, 20)
    assert q4k.matmul_grouped_combine(w, x, r).shape == (0, 20)
    full = q4k.moe_route(torch.zeros((4, 3), device=dev), 2)
    assert q4k.matmul_grouped(w[:, :0].contiguous(), torch.zeros((4, 256), device=dev), full.offsets, full.rows,
                              x_div=2).shape == (8, 0)
    # groups that are all empty: no row is written
    y = torch.full((8, 20), 7.0, device=dev)
    q4k.matmul_grouped(w, torch.zeros((4, 256), device=dev), r.offsets, full.rows, y=y, x_div=2)
    assert bool((y == 7.0).all())


@pytest.mark.parametrize("sizes", [[2, 1], [40, 3], [200, 9]], ids=str)
def test_unusual_activations(sizes):
    """Zero rows, tiny and huge magnitudes, and a row with NaN or infinity, which
    must not reach any other row."""
    import torch
    offsets, rows, P = _table(sizes, 10)
    N, K = 48, 1024
    w, x = _weights(2, N, K, 7), qi.random_x(P, K, seed=10)
    x[0] = 0.0
    x[1] *= np.float32(1e-36)
    x[2] *= np.float32(1e30)
    y = q4k.matmul_grouped(to_dev(w), to_dev(x), to_dev(offsets), to_dev(rows)).cpu().numpy()
    want, s = ref.grouped(w, x, offsets, rows, 1, P)
    assert np.all(y[0] == 0.0)
    # sums of products below 2^-126 may lose their low bits
    err = np.abs(y.astype(np.float64) - want)
    assert np.all(err <= ref.product_tol(K) * s + K * 2.0 ** -149)
    bad = x.copy()
    bad[1, 5] = np.nan
    bad[2, 7] = np.inf
    z = q4k.matmul_grouped(to_dev(w), to_dev(bad), to_dev(offsets), to_dev(rows)).cpu().numpy()
    assert not np.isfinite(z[1]).any() and not np.isfinite(z[2]).any()
    other = np.setdiff1d(np.arange(P), [1, 2])
    assert np.array_equal(z[other], y[other])


def test_one_hot_rows_give_the_weights():
    """x = a unit vector: the products are single weights, which the two-term
    form returns within two roundings."""
    import torch
    E, N, K = 3, 40, 512
    w = _weights(E, N, K, 8)
    at = _rng(11).integers(0, K, 60)
    x = qi.one_hot_x(60, K, at)
    offsets = np.array([0, 2, 22, 60], np.int32)
    y = q4k.matmul_grouped(to_dev(w), to_dev(x), to_dev(offsets)).cpu().numpy()
    for e in range(E):
        val, mag = ref.unpack(w[e])
        r = np.arange(offsets[e], offsets[e + 1])
        assert np.all(np.abs(y[r] - val[:, at[r]].T) <= 2 * 2.0 ** -24 * mag[:, at[r]].T)


def test_results_do_not_depend_on_the_run():
    """The same call twice gives the same bits."""
    sizes = [70, 3, 0, 18]
    offsets, rows, P = _table(sizes, 12)
    w, x = to_dev(_weights(4, 90, 1024, 9)), to_dev(qi.random_x(P, 1024, seed=12))
    import torch
    a = q4k.matmul_grouped(w, x, to_dev(offsets), to_dev(rows))
    b = q4k.matmul_grouped(w, x, to_dev(offsets), to_dev(rows))
    assert torch.equal(a, b)


def test_weights_behind_four_gigabytes():
    """The last expert's matrix starts past 2^32 bytes."""
    import torch
    E, N, K = 33, 30000, 8192
    row = K // 256 * 144
    assert (E - 1) * N * row > 1 << 32
    w = torch.zeros((E, N, row), dtype=torch.uint8, device=device())
    last = qi.random_q4k(64, K, seed=13)
    w[E - 1, N - 64:] = to_dev(last)
    x = qi.random_x(3, K, seed=13)
    offsets = np.zeros(E + 1, np.int32)
    offsets[-1] = 3
    y = q4k.matmul_grouped(w, to_dev(x), to_dev(offsets)).cpu().numpy()
    want, s = ref.grouped(last[None], x, [0, 3], np.arange(3), 1, 3)
    check_close(y[:, -64:], want, s, ref.product_tol(K))
    assert np.all(y[:, :-64] == 0.0)


def test_outputs_behind_two_to_the_31():
    """The last rows of y start past 2^31 elements; rows in between are left alone."""
    import torch
    E, N, K, P = 2, 32768, 256, 66000
    w = _weights(E, N, K, 15)
    x = qi.random_x(P, K, seed=15)
    y = torch.full((P, N), 7.0, device=device())
    offsets = np.array([0, 3, 40], np.int32)
    rows = np.concatenate([[0, 5, P - 1], np.arange(P - 38, P - 1)]).astype(np.int32)
    rows = np.concatenate([rows, np.full(P - 40, -1, np.int32)])
    assert (P - 1) * N > 1 << 31
    q4k.matmul_grouped(to_dev(w), to_dev(x), to_dev(offsets), to_dev(rows), y=y)
    for e in range(E):
        r = rows[offsets[e]:offsets[e + 1]]
        val, mag = ref.unpack(w[e])
        xs = x[r].astype(np.float64)
        check_close(y[torch.from_numpy(r.astype(np.int64)).to(y.device)].cpu().numpy(), xs @ val.T, np.abs(xs) @ mag.T,
                    ref.product_tol(K))
    assert bool((y[1:5] == 7.0).all()) and bool((y[6:P - 38] == 7.0).all())


# ---- a layer of them ---------------------------------------------------------------

def _layer(M, E, k, hidden, ffn, tag):
    g = _rng(20, tag)
    d = dict(d_range=(1e-4, 4e-4), dmin_range=(1e-3, 3e-3))
    return dict(
        logits=(1.5 * g.standard_normal((M, E))).astype(np.float32),
        x=qi.random_x(M, hidden, seed=qi.tensor_seed(qi.BASE_SEED, 1120, tag)),
        gate=np.stack([qi.random_q4k(ffn, hidden, qi.tensor_seed(1, tag, e), **d) for e in range(E)]),
        up=np.stack([qi.random_q4k(ffn, hidden, qi.tensor_seed(2, tag, e), **d) for e in range(E)]),
        down=np.stack([qi.random_q4k(hidden, ffn, qi.tensor_seed(3, tag, e), **d) for e in range(E)]))


def _run_layer(t, k):
    r = q4k.moe_route(t["logits"], k)
    h = q4k.matmul_grouped_swiglu(t["gate"], t["up"], t["x"], r.offsets, r.rows, x_div=k)
    return q4k.matmul_grouped_combine(t["down"], h, r)


@pytest.mark.parametrize("M,E,k,hidden,ffn", [(1, 16, 4, 512, 256), (7, 8, 2, 256, 512), (150, 12, 3, 512, 256)])
def test_layer(M, E, k, hidden, ffn):
    c = _layer(M, E, k, hidden, ffn, M)
    t = {n: to_dev(v) for n, v in c.items()}
    got = _run_layer(t, k).cpu().numpy().astype(np.float64)
    expert, weight = ref.route(c["logits"], None, k, False, True, 1.0)
    want = np.zeros((M, hidden))
    scale = np.zeros((M, hidden))
    W = {n: [ref.unpack(c[n][e]) for e in range(E)] for n in ("gate", "up", "down")}
    x = c["x"].astype(np.float64)
    for m in range(M):
        for j in range(k):
            e = expert[m, j]
            g, u = W["gate"][e][0] @ x[m], W["up"][e][0] @ x[m]
            gs, us = W["gate"][e][1] @ np.abs(x[m]), W["up"][e][1] @ np.abs(x[m])
            h = ref.silu(g) * u
            # h carries the error of its two products, bounded as in test_grouped_swiglu
            hs = np.abs(h) * (1 + np.abs(g)) + 1.1 * gs * np.abs(u) + np.abs(ref.silu(g)) * us
            want[m] += weight[m, j] * (W["down"][e][0] @ h)
            scale[m] += weight[m, j] * (W["down"][e][1] @ (np.abs(h) + hs))
    # first order: each factor is off by at most product_tol of its own scale
    tol = 2 * ref.product_tol(max(hidden, ffn)) + 64 * 2.0 ** -23
    err = np.abs(got - want)
    assert np.all(err <= tol * scale), (err / scale).max()


@pytest.mark.parametrize("M", [1, 5, 150])
def test_layer_captured_and_replayed(M):
    """One graph of the whole layer, replayed on changing inputs with eager work
    of the same program between the replays."""
    import torch
    k = 3
    c = _layer(M, 12, k, 512, 256, 77)
    t = {n: to_dev(v) for n, v in c.items()}
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        _run_layer(t, k)  # grows the workspace before the capture
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        out = _run_layer(t, k)
    for step in range(4):
        t["x"].copy_(to_dev(qi.random_x(M, 512, seed=100 + step)))
        t["logits"].copy_(to_dev(_rng(30, step).standard_normal(c["logits"].shape).astype(np.float32)))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        want = _run_layer(t, k)  # eager, on the default stream
        torch.cuda.synchronize()
        assert torch.equal(got, want), step


def test_two_streams_at_once():
    import torch
    k = 2
    ts = []
    for tag, M in ((41, 90), (42, 4)):
        ts.append({n: to_dev(v) for n, v in _layer(M, 6, k, 512, 256, tag).items()})
    want = [_run_layer(t, k) for t in ts]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ts]
    for _ in range(5):
        got = []
        for t, s in zip(ts, streams):
            with torch.cuda.stream(s):
                got.append(_run_layer(t, k))
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_layer_from_a_gguf_tensor(tmp_path):
    """A 3-D expert tensor of a GGUF file, uploaded by load_q4k, viewed per expert."""
    from tests.gguf_writer import write_gguf
    E, N, K = 3, 20, 256
    w = _weights(E, N, K, 14)
    path = tmp_path / "experts.gguf"
    write_gguf(path, [], [("ffn_up_exps.weight", q4k.GGUF_TYPE_Q4_K, (K, N, E), w.tobytes())])
    wd = q4k.load_q4k(path)["ffn_up_exps.weight"].view(E, N, -1)
    x = qi.random_x(9, K, seed=14)
    offsets = np.array([0, 4, 4, 9], np.int32)
    y = q4k.matmul_grouped(wd, to_dev(x), to_dev(offsets)).cpu().numpy()
    want, s = ref.grouped(w, x, offsets, np.arange(9), 1, 9)
    check_close(y, want, s, ref.product_tol(K))
