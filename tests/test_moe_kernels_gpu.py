"""Every kernel of the grouped products (include/q4k_moe.h) on the inputs where one
can go wrong.  The sizes below name the kernel that they are meant for, and a
test that needs no GPU asserts that they reach it, so a change of the rule that
chooses cannot leave a kernel untested."""
import ctypes

import numpy as np
import pytest

import gguf_q4_dequant_amd as q4k
import q4k_inputs as qi
from tests import moe_reference as ref
from tests.gpu_helpers import check_close, device, to_dev

gpu = pytest.mark.gpu

# (rows of a tile, parts of K, gate/up form): (group sizes, N, K).  Odd numbers of
# super-blocks, so that a split of K ends unevenly, and enough of them for every
# buffer to be filled again; columns that end one behind a workgroup's; groups
# whose last tile holds one, two and three sixteens of rows, one empty group.
KERNELS = {
    (4, 4, False): ([3, 0, 17, 20], 289, 1024),
    (4, 4, True): ([3, 0, 17, 20], 289, 768),
    (4, 8, False): ([1, 2, 30, 7], 33, 2304),
    (4, 8, True): ([1, 2, 30, 7], 129, 4352),
    (16, 4, False): ([90, 0, 33, 77], 897, 1792),
    (16, 4, True): ([90, 0, 33, 77], 449, 2816),
    (16, 2, False): ([201, 0, 152, 131], 897, 1280),
    (16, 2, True): ([130, 0, 71, 99], 961, 2304),
    (16, 1, False): ([3, 17, 0, 8, 16, 1] * 4, 2689, 1280),
    (16, 1, True): ([3, 17, 0, 8, 16, 1] * 4, 1345, 1792),
    (32, 1, False): ([290, 0, 307, 411], 2049, 2304),
    (32, 1, True): ([290, 0, 307, 411], 1025, 1280),
    (48, 1, False): ([48 * 20 + 7, 0, 48 * 41 + 30, 48 * 23 + 41], 3329, 1280),
    (48, 1, True): ([48 * 20 + 7, 0, 48 * 41 + 30, 48 * 23 + 41], 1665, 2304),
}
PLAIN = [k for k in KERNELS if not k[2]]
name = lambda k: f"{k[0]}rows-{k[1]}parts" + ("-swiglu" if k[2] else "")  # noqa: E731
kernels = pytest.mark.parametrize("kernel", list(KERNELS), ids=name)
plain_kernels = pytest.mark.parametrize("kernel", PLAIN, ids=name)


def test_the_sizes_reach_the_kernels_they_name():
    assert {k[:2] for k in PLAIN} == {k[:2] for k in KERNELS if k[2]} == \
        {(4, 4), (4, 8), (16, 1), (16, 2), (16, 4), (32, 1), (48, 1)}
    for (rows, parts, swiglu), (sizes, N, K) in KERNELS.items():
        got = q4k.grouped_tile(len(sizes), sum(sizes), N, K, swiglu)
        assert got == (rows, parts), (rows, parts, swiglu, got)


def test_tile_query():
    lib = q4k.library()
    for bad in ((0, 8, 16, 256), (1025, 8, 16, 256), (4, -1, 16, 256), (4, 8, -1, 256), (4, 8, 16, 0), (4, 8, 16, 300),
                (4, 8, 16, -256), (4, 8, 16, 2 ** 26 + 256)):
        parts = ctypes.c_int(5)
        assert lib.q4k_grouped_tile(*bad, 0, ctypes.byref(parts)) == q4k.ERR_BAD_DIM and parts.value == 0, bad
        with pytest.raises(q4k.Q4KError):
            q4k.grouped_tile(*bad)
    assert lib.q4k_grouped_tile(4, 8, 16, 256, 1, None) in (4, 16, 32, 48)
    assert q4k.grouped_tile(4, 0, 16, 256) == (0, 0) and q4k.grouped_tile(4, 8, 0, 256) == (0, 0)


# ---- the products --------------------------------------------------------------

def _rng(*path):
    return np.random.Generator(np.random.PCG64(qi.tensor_seed(qi.BASE_SEED, 1300, *path)))


def _weights(E, N, K, tag, **ranges):
    return np.stack([qi.random_q4k(N, K, qi.tensor_seed(qi.BASE_SEED, 1301, tag, e, N, K), **ranges) for e in range(E)])


def _case(kernel, tag, x_div=1, scale=0.02, **ranges):
    """Matrices, x, and a table whose pairs come in a random order."""
    sizes, N, K = KERNELS[kernel]
    P, E = sum(sizes), len(sizes)
    rows = _rng(tag, P).permutation(P).astype(np.int32)
    offsets = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    w = [_weights(E, N, K, 10 * tag + i, **ranges) for i in range(2 if kernel[2] else 1)]
    x = (scale * qi.random_x((P + x_div - 1) // x_div, K, qi.tensor_seed(qi.BASE_SEED, 1302, tag, P, K))).astype(np.float32)
    return w, x, offsets, rows, P, N, K


def _run(kernel, w, x, offsets, rows, x_div=1, y=None):
    if kernel[2]:
        return q4k.matmul_grouped_swiglu(w[0], w[1], x, offsets, rows, out=y, x_div=x_div)
    return q4k.matmul_grouped(w[0], x, offsets, rows, y=y, x_div=x_div)


def _check(kernel, got, w, x, offsets, rows, x_div, P, K):
    """Against the 64-bit form; rows that no group names are returned, not compared."""
    want, s = ref.grouped(w[0], x, offsets, rows, x_div, P)
    named = ~np.isnan(want[:, 0])
    got, want, s = got[named].astype(np.float64), want[named], s[named]
    if not kernel[2]:
        check_close(got, want, s, ref.product_tol(K))
        return named
    u, su = (a[named] for a in ref.grouped(w[1], x, offsets, rows, x_div, P))
    # |silu'| < 1.1; the exponential's argument carries |g| * 2^-23, the rest a few ulp
    t = ref.product_tol(K)
    bound = 1.1 * t * s * (np.abs(u) + t * su) + np.abs(ref.silu(want)) * t * su + \
        np.abs(ref.silu(want) * u) * (np.abs(want) + 8) * 2.0 ** -23
    err = np.abs(got - ref.silu(want) * u)
    assert np.all(err <= bound + 1e-30), (err / (bound + 1e-30)).max()
    return named


@gpu
@kernels
def test_product_over_every_buffer(kernel):
    """x of one row for two pairs, entries outside [0, P) inside the groups."""
    import torch
    w, x, offsets, rows, P, N, K = _case(kernel, 1, x_div=2)
    for at, entry in ((0, -1), (int(offsets[2]) + 1, P), (P - 1, np.iinfo(np.int32).max), (P // 2, np.iinfo(np.int32).min)):
        rows[at] = entry
    y = torch.full((P, N), 7.0, device=device())
    wd, args = [to_dev(a) for a in w], (to_dev(x), to_dev(offsets), to_dev(rows))
    _run(kernel, wd, *args, x_div=2, y=y)
    got = y.cpu().numpy()
    named = _check(kernel, got, w, x, offsets, rows, 2, P, K)
    assert (~named).sum() == 4 and np.all(got[~named] == 7.0)
    # the same call again: the same bits
    again = _run(kernel, wd, *args, x_div=2, y=torch.full((P, N), 7.0, device=device()))
    assert torch.equal(again, y)


@gpu
@plain_kernels
def test_unusual_rows_on_every_kernel(kernel):
    """Zero rows, tiny and huge magnitudes, and rows with NaN or infinity, which
    share tiles with others and must not reach them."""
    w, x, offsets, rows, P, N, K = _case(kernel, 2, scale=1.0)
    r = rows[:8] if P < 300 else rows[[0, 1, 2, 20, 40, 47, 48, int(offsets[1]) - 1]]
    zero, tiny, huge, mixed, nan, inf, ninf, both = r
    x[zero] = 0.0
    x[tiny] *= np.float32(1e-36)
    x[huge] *= np.float32(1e30)
    x[mixed, ::3] *= np.float32(1e-20)   # small values beside ordinary ones
    wd, args = [to_dev(a) for a in w], (to_dev(offsets), to_dev(rows))
    y = _run(kernel, wd, to_dev(x), *args).cpu().numpy()
    want, s = ref.grouped(w[0], x, offsets, rows, 1, P)
    assert np.all(y[zero] == 0.0)
    err = np.abs(y.astype(np.float64) - want)
    # sums of products below 2^-126 may lose their low bits
    assert np.all(err <= ref.product_tol(K) * s + K * 2.0 ** -149), (err / np.maximum(s, 1e-300)).max()
    bad = x.copy()
    bad[nan, 5] = np.nan
    bad[inf, K - 1] = np.inf
    bad[ninf, K // 2] = -np.inf
    bad[both, 0], bad[both, 300] = np.nan, np.inf
    z = _run(kernel, wd, to_dev(bad), *args).cpu().numpy()
    hit = np.array([nan, inf, ninf, both])
    assert not np.isfinite(z[hit]).any()
    other = np.setdiff1d(np.arange(P), hit)
    assert np.array_equal(z[other], y[other])


@gpu
@plain_kernels
def test_single_weights_on_every_kernel(kernel):
    """x = unit vectors: the products are single weights."""
    w, x, offsets, rows, P, N, K = _case(kernel, 3)
    at = _rng(4, P).integers(0, K, P)
    x = qi.one_hot_x(P, K, at)
    y = _run(kernel, [to_dev(a) for a in w], to_dev(x), to_dev(offsets), to_dev(rows)).cpu().numpy()
    for e in range(len(offsets) - 1):
        r = rows[offsets[e]:offsets[e + 1]]
        val, mag = ref.unpack(w[0][e])
        assert np.all(np.abs(y[r] - val[:, at[r]].T) <= 2 * 2.0 ** -24 * mag[:, at[r]].T)


@gpu
@pytest.mark.parametrize("holes", [False, True])
@plain_kernels
def test_weighted_sum_behind_every_kernel(kernel, holes):
    """The products of the weighted sum use both slots of the workspace."""
    sizes, N, K = KERNELS[kernel]
    E, k = len(sizes), 2
    M = sum(sizes) // k
    assert q4k.grouped_tile(E, M * k, N, K) == kernel[:2]
    g = _rng(5, M, E)
    expert = np.argsort(g.random((M, E)) + np.arange(E) * 0.2, axis=1)[:, :k].astype(np.int32)
    if holes:
        expert[g.random((M, k)) < 0.3] = -1
        expert[M // 2] = -1
    weight = g.random((M, k)).astype(np.float32)
    offsets, rows = ref.stable_groups(expert, E)
    w = _weights(E, N, K, 50)
    x = qi.random_x(M * k, K, qi.tensor_seed(qi.BASE_SEED, 1303, M, K))
    r = q4k.Routing(to_dev(expert), to_dev(weight), to_dev(offsets), to_dev(rows))
    out = q4k.matmul_grouped_combine(to_dev(w), to_dev(x), r).cpu().numpy()
    y, s = ref.grouped(w, x, offsets, rows[:offsets[-1]], 1, M * k)
    y, s = np.nan_to_num(y).reshape(M, k, N), np.nan_to_num(s).reshape(M, k, N)
    want = (weight[:, :, None].astype(np.float64) * y).sum(1)
    # the products' error, and k fused multiply-adds of at most 2^-24 of sum |weight| |y| each
    bound = (weight[:, :, None] * s).sum(1) * (ref.product_tol(K) + k * 2.0 ** -24)
    err = np.abs(out.astype(np.float64) - want)
    assert np.all(err <= bound), (err / np.maximum(bound, 1e-30)).max()
    if holes:
        assert np.all(out[M // 2] == 0.0)


@gpu
@plain_kernels
def test_rows_up_to_the_largest_float(kernel):
    """Finite rows give finite products, whatever their magnitude: maxima around
    the largest that one power of two brings into binary16, and the largest float."""
    small = dict(d_range=(1e-6, 2e-6), dmin_range=(0.0, 4e-6))  # no sum of magnitudes reaches 2^128
    w, x, offsets, rows, P, N, K = _case(kernel, 6, scale=1.0, **small)
    top = np.finfo(np.float32).max
    magnitudes = [top, 1e38, 2.0 ** 127, 6.7e35, 65520.0 * 2.0 ** 103, np.nextafter(np.float32(2.0 ** 118), np.float32(0)), 1e36]
    shaped = rows[:len(magnitudes)] if P < 300 else rows[[0, 1, 20, 40, 47, 48, int(offsets[1]) - 1]]
    for row, m in zip(shaped, magnitudes):
        shape = x[row].astype(np.float64) / np.abs(x[row]).max()
        x[row] = shape * float(m)
        assert np.abs(x[row]).max() == np.float32(m)
    y = _run(kernel, [to_dev(a) for a in w], to_dev(x), to_dev(offsets), to_dev(rows)).cpu().numpy()
    want, s = ref.grouped(w[0], x, offsets, rows, 1, P)
    assert s.max() < top and np.isfinite(y).all()
    check_close(y, want, s, ref.product_tol(K))


@gpu
@pytest.mark.parametrize("kernel", [k for k in KERNELS if k[2]], ids=name)
def test_swiglu_of_the_largest_floats(kernel):
    """A gate of zeros: silu(0) * u is 0 for every finite u."""
    w, x, offsets, rows, P, N, K = _case(kernel, 7, scale=1.0, d_range=(1e-6, 2e-6), dmin_range=(0.0, 4e-6))
    # the largest float in every seventh place: over all K = 4352 places the sum of
    # magnitudes would be 7.2e38, above the largest float; over these it is 1.0e38
    x[rows[0], ::7], x[rows[P - 1]] = np.finfo(np.float32).max, -1e36
    w[0][:] = 0
    out = _run(kernel, [to_dev(a) for a in w], to_dev(x), to_dev(offsets), to_dev(rows)).cpu().numpy()
    u, s = ref.grouped(w[1], x, offsets, rows, 1, P)
    assert s.max() < np.finfo(np.float32).max and np.all(out == 0.0)


@gpu
@plain_kernels
def test_small_values_beside_a_large_one(kernel):
    """Each value of a row is kept to 2^-22 of itself or 2^-39 of the row's largest
    magnitude, and each sum of 32 (the min term) to 2^-33 of that magnitude: one
    large value where W is zero, and one small value elsewhere.  The large one is
    2^14, which is not scaled; then both limits are half of a binary16's smallest
    step, 2^-25, the second times the 2^6 that the sums are divided by."""
    w, x, offsets, rows, P, N, K = _case(kernel, 8)
    blocks = w[0].reshape(len(offsets) - 1, N, K // 256, 144)
    blocks[:, :, 0, :4] = 0  # d and dmin of the first super-block
    g = _rng(9, P)
    at, v = g.integers(256, K, P), (g.choice([-1, 1], P) * g.uniform(2.0 ** -4, 2.0 ** -3, P)).astype(np.float32)
    x[:] = 0.0
    x[:, 17] = 2.0 ** 14
    x[np.arange(P), at] = v
    y = _run(kernel, [to_dev(a) for a in w], to_dev(x), to_dev(offsets), to_dev(rows)).cpu().numpy().astype(np.float64)
    for e in range(len(offsets) - 1):
        r = rows[offsets[e]:offsets[e + 1]]
        val, mag = ref.unpack(w[0][e])
        least = (mag - val)[:, at[r]].T / 2   # dmin * m
        scaled = (mag + val)[:, at[r]].T / 2  # d * sc * q
        v64 = np.abs(v[r].astype(np.float64))[:, None]
        bound = (2.0 ** -22 * v64 + 2.0 ** -25) * scaled + (2.0 ** -22 * v64 + 2.0 ** -19) * least
        # two products, their factors and the last sum, each off by at most 2^-24 of the two terms
        bound += 8 * 2.0 ** -24 * v64 * (scaled + least)
        err = np.abs(y[r] - v[r].astype(np.float64)[:, None] * val[:, at[r]].T)
        assert np.all(err <= bound), (err / np.maximum(bound, 1e-300)).max()


# ---- a layer of them: graphs and streams -------------------------------------------

# rows of a tile: (M, E, top_k, hidden, ffn), both products of the layer on that kernel
LAYERS = {4: (5, 12, 3, 512, 256), 16: (200, 8, 2, 1024, 512), 32: (600, 4, 2, 1280, 1280), 48: (2600, 4, 2, 2560, 1280)}
layers = pytest.mark.parametrize("tile", list(LAYERS), ids=lambda t: f"{t}rows")


def test_the_layers_reach_the_kernels_they_name():
    for tile, (M, E, k, hidden, ffn) in LAYERS.items():
        got = q4k.grouped_tile(E, M * k, ffn, hidden, True)[0], q4k.grouped_tile(E, M * k, hidden, ffn)[0]
        assert got == (tile, tile), (tile, got)


def _layer(tile, tag):
    M, E, k, hidden, ffn = LAYERS[tile]
    g = _rng(20, tile, tag)
    small = dict(d_range=(1e-4, 4e-4), dmin_range=(1e-3, 3e-3))
    return {n: to_dev(v) for n, v in dict(
        logits=(1.5 * g.standard_normal((M, E))).astype(np.float32),
        x=qi.random_x(M, hidden, qi.tensor_seed(qi.BASE_SEED, 1320, tile, tag)),
        gate=_weights(E, ffn, hidden, 100 * tag + 1, **small), up=_weights(E, ffn, hidden, 100 * tag + 2, **small),
        down=_weights(E, hidden, ffn, 100 * tag + 3, **small)).items()}, k


@pytest.fixture(scope="module")
def streams():
    """Two streams for all (torch hands out the same 32 in turn)."""
    import torch
    return torch.cuda.Stream(), torch.cuda.Stream()


def _run_layer(t, k):
    r = q4k.moe_route(t["logits"], k)
    h = q4k.matmul_grouped_swiglu(t["gate"], t["up"], t["x"], r.offsets, r.rows, x_div=k)
    return q4k.matmul_grouped_combine(t["down"], h, r)


@gpu
@layers
def test_graphs_that_share_a_workspace(tile, streams):
    """Two layers captured on one stream, replayed in turn on changing inputs with
    eager work of the same program between the replays."""
    import torch
    stream = streams[0]
    stream.wait_stream(torch.cuda.current_stream())
    parts = [_layer(tile, tag) for tag in (1, 2)]
    with torch.cuda.stream(stream):
        for t, k in parts:
            _run_layer(t, k)  # grows the workspace before the captures
    torch.cuda.synchronize()
    graphs = []
    for t, k in parts:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            out = _run_layer(t, k)
        graphs.append((graph, out))
    for step in range(3):
        for i, (t, k) in enumerate(parts):
            t["x"].copy_(to_dev(qi.random_x(*t["x"].shape, seed=200 + 10 * step + i)))
            t["logits"].copy_(to_dev(_rng(30, step, i).standard_normal(tuple(t["logits"].shape)).astype(np.float32)))
        torch.cuda.synchronize()
        for graph, _ in graphs:
            graph.replay()
        torch.cuda.synchronize()
        for (t, k), (_, out) in zip(parts, graphs):
            assert torch.equal(out, _run_layer(t, k)), step


@gpu
@layers
def test_layers_on_two_streams_at_once(tile, streams):
    import torch
    parts = [_layer(tile, tag) for tag in (3, 4)]
    want = [_run_layer(t, k) for t, k in parts]
    torch.cuda.synchronize()
    for _ in range(4):
        got = []
        for (t, k), s in zip(parts, streams):
            with torch.cuda.stream(s):
                got.append(_run_layer(t, k))
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
