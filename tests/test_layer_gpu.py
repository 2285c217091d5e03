"""The operators of include/q4k_layer.h together with the packed products, as a decoder
layer runs them: prompts, single tokens, drafted tokens and the accepted ones stored
again; captured graphs, other streams, calls after one another on one workspace."""
import threading

import numpy as np
import pytest

import gguf_q4_dequant_amd as q4k
import oracle
import q4k_inputs as qi
from tests.gpu_helpers import to_dev
from tests.layer_reference import Paged, attention, rng_of, rotation, tolerance

pytestmark = pytest.mark.gpu

H, HQ, HK, D, F, PAGE = 512, 8, 2, 64, 768, 16
EPS = 1e-6


def weights():
    """A layer's packed matrices, about centred and of size 1 / sqrt(K), its norms and the rotation."""
    out = {}
    for i, (name, n, k) in enumerate([("q", HQ * D, H), ("k", HK * D, H), ("v", HK * D, H), ("o", H, HQ * D),
                                      ("gate", F, H), ("up", F, H), ("down", H, F)]):
        d = 1 / (200 * np.sqrt(k))
        out[name] = qi.random_q4k(n, k, seed=qi.tensor_seed(qi.BASE_SEED, 1600, i), d_range=(0.5 * d, 1.5 * d),
                                  dmin_range=(4 * d, 11 * d))
    rng = rng_of(50)
    for name, n in (("norm1", H), ("norm2", H), ("q_norm", D), ("k_norm", D)):
        out[name] = (0.5 + rng.random(n)).astype(np.float32)
    out["inv_freq"] = (10000.0 ** (-np.arange(D // 2) / (D // 2))).astype(np.float32)
    return out


def device_layer(w, x, cache, seqs, positions=None, mask=None):
    """One layer on the GPU: x [T, H] -> x [T, H], and its keys and values."""
    T = x.shape[0]
    h = q4k.rms_norm(x, w["norm1"], EPS)
    q, k, v = (x.new_empty(T, n * D) for n in (HQ, HK, HK))
    q4k.matmul_batched([(w["q"], h, q), (w["k"], h, k), (w["v"], h, v)])
    k, v = k.view(T, HK, D), v.view(T, HK, D)
    q = q4k.kv_append(k, v, cache, seqs, rotation=q4k.Rotation(w["inv_freq"]), q=q.view(T, HQ, D), positions=positions,
                      q_norm=w["q_norm"], k_norm=w["k_norm"], eps=EPS)
    o = q4k.attention(q, cache, seqs) if mask is None else q4k.attention_tree(q, cache, seqs, mask)
    h, x = q4k.rms_norm(q4k.matmul(w["o"], o.view(T, HQ * D)), w["norm2"], EPS, residual=x)
    return x + q4k.matmul(w["down"], q4k.matmul_swiglu(w["gate"], w["up"], h)), k, v


class PlainLayer:
    """The same in 64 bits; a sequence's keys and values by index, not rounded."""

    def __init__(self, w, sequences):
        K = {"o": HQ * D, "down": F}
        self.m = {n: oracle.dequant_exact(w[n], K.get(n, H)).reshape(-1, K.get(n, H)) for n in ("q", "k", "v", "o", "gate", "up", "down")}
        self.w, self.kv = w, [([], []) for _ in range(sequences)]

    def __call__(self, x, rows, positions, see):
        """rows: (sequence, index) of every row; see(t): the indexes that row t sees."""
        norm = lambda t, g: t / np.sqrt((t * t).mean(-1, keepdims=True) + EPS) * g  # noqa: E731
        T = len(rows)
        h = norm(x, self.w["norm1"])
        q, k, v = (h @ self.m[n].T for n in ("q", "k", "v"))
        q, _ = rotation(q.reshape(T, HQ, D), self.w["q_norm"], EPS, positions, self.w["inv_freq"], False)
        k, _ = rotation(k.reshape(T, HK, D), self.w["k_norm"], EPS, positions, self.w["inv_freq"], False)
        for t, (b, j) in enumerate(rows):
            for store, value in zip(self.kv[b], (k[t], v.reshape(T, HK, D)[t])):
                store[j:j + 1] = [value]
        o = np.zeros((T, HQ, D))
        for t, (b, _) in enumerate(rows):
            K, V = (np.array([s[j] for j in see(t)]) for s in self.kv[b])
            for head in range(HQ):
                s = K[:, head // (HQ // HK)] @ q[t, head] / np.sqrt(D)
                p = np.exp(s - s.max())
                o[t, head] = p / p.sum() @ V[:, head // (HQ // HK)]
        x = x + o.reshape(T, -1) @ self.m["o"].T
        h = norm(x, self.w["norm2"])
        g = h @ self.m["gate"].T
        return x + (g / (1 + np.exp(-g)) * (h @ self.m["up"].T)) @ self.m["down"].T


def check(got, want):
    """Keys, values and their products: the cache's rounding (2^-11 of each) moves a score by about
    2^-11 |q| |k| / sqrt(D) ~ 2^-9 at |q| |k| / sqrt(D) = 4 or less, a weighted value by as much and 2^-11;
    the products (at most 16 rows) are exact to 1e-5 of sum |x w| (about 20 of the result's size): 2e-4 each.
    Half of a row's size comes from x itself; 2^-8 of the largest value covers the sum."""
    got = got.cpu().numpy()
    assert np.abs(got - want).max() <= 2.0 ** -8 * np.abs(want).max()


def test_prompts_tokens_drafts_and_accepted_drafts():
    import torch
    w = weights()
    dev = {n: to_dev(a) for n, a in w.items()}
    plain = PlainLayer(w, 2)
    rng = rng_of(51)
    i32 = lambda a: to_dev(np.asarray(a, np.int32))  # noqa: E731
    pages = i32([[3, 0, 5], [1, 4, 2]])
    pool = torch.full((6, HK, PAGE, D), float("nan"), dtype=torch.float16, device="cuda")
    cache = q4k.KVCache(pool, pool.clone())
    lengths = np.array([0, 0])

    def step(n, positions=None, mask=None):
        """n[b] new tokens of each sequence, random inputs; returns keys and values."""
        nonlocal lengths
        before, lengths = lengths, lengths + n
        rows = [(b, int(before[b]) + i) for b in range(2) for i in range(n[b])]
        x = rng.standard_normal((len(rows), H)).astype(np.float32)
        seqs = q4k.Sequences(i32([0, n[0], n[0] + n[1]]), i32(lengths), pages)
        pos = np.array([j for _, j in rows] if positions is None else positions)
        if mask is None:
            see = lambda t: range(rows[t][1] + 1)  # noqa: E731
        else:
            see = lambda t: [j for j in range(int(lengths[rows[t][0]]))  # noqa: E731
                             if j < before[rows[t][0]] or mask[t] >> (j - int(before[rows[t][0]])) & 1]
        got, k, v = device_layer(dev, to_dev(x), cache, seqs, None if positions is None else i32(positions),
                                 None if mask is None else i32(mask).view(-1, 1))
        check(got, plain(x.astype(np.float64), rows, pos, see))
        return k, v, pos

    step((9, 7))
    for _ in range(3):
        step((1, 1))
    # drafts: 0 -> 1 -> 2 and 0 -> 3 in the first sequence; 0 and 1 -> 2 in the second
    base = lengths.copy()
    depth = np.array([0, 1, 2, 1, 0, 0, 1])
    k, v, pos = step((4, 3), np.repeat(base, (4, 3)) + depth, [1, 3, 7, 9, 1, 2, 6])
    # accepted: 0 -> 3 and 1 -> 2, stored again where they belong (their values are as they were)
    keep = [0, 3, 5, 6]
    seqs = q4k.Sequences(i32([0, 2, 4]), i32(base + 2), pages)
    q4k.kv_append(k[keep], v[keep], cache, seqs, rotation=q4k.Rotation(dev["inv_freq"]), k_norm=dev["k_norm"], eps=EPS)
    for b, (first, rows) in enumerate(((0, (0, 3)), (0, (1, 2)))):
        for store in plain.kv[b]:
            store[base[b]:] = [store[base[b] + r] for r in rows]
    lengths = base + 2
    assert pos[3] == base[0] + 1 and pos[6] == base[1] + 1  # the depths are the places
    step((1, 1))
    step((2, 3))


def _decode(rng, kind="f16", sizes=((70, 1), (5, 1), (300, 1))):
    p = Paged(rng, list(sizes), 2, 64, 16, kind, extra_cols=2)
    return p, rng.standard_normal((p.T, 8, 64)).astype(np.float32)


def test_graph_replays():
    """A captured step (norm, rotation and append, attention split along the keys, a tree, a
    prompt chunk) gives the eager bits for new lengths, pages, queries and keys, replay after replay."""
    import torch
    rng = rng_of(60)
    p, q = _decode(rng, sizes=((900, 1), (40, 1), (1500, 1)))
    cache, seqs = p.on_device()
    t, tq = _decode(rng, sizes=((800, 12), (30, 40)))
    tcache, tseqs = t.on_device()
    mask = to_dev(rng.integers(0, 2 ** 31, (t.T, 2), dtype=np.int32))
    x, w = torch.randn(3, 512, device="cuda"), torch.rand(512, device="cuda")
    q, tq, k = to_dev(q), to_dev(tq), torch.randn(3, 2, 64, device="cuda")
    rot = q4k.Rotation(torch.rand(32, device="cuda"))

    def step():
        y, total = q4k.rms_norm(x, w, residual=x)
        turned = q4k.kv_append(k, k, cache, seqs, rotation=rot, q=q)
        return (y, total, turned, q4k.attention(turned, cache, seqs), q4k.attention(tq, tcache, tseqs),
                q4k.attention_tree(tq, tcache, tseqs, mask))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
        side.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            outs = step()
    torch.cuda.synchronize()
    for rep in range(4):
        for a in (x, q, tq, k):
            a.copy_(torch.randn_like(a))
        seqs.lengths.copy_(to_dev(np.array([(901, 41, 1501), (1, 2, 3), (500, 0, 17), (901, 41, 1501)][rep], np.int32)))
        seqs.pages[0, :4] = seqs.pages[0, torch.randperm(4)]
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in outs]
        junk = torch.randn(1 << 20, device="cuda").sum()
        want = step()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b), rep
        del junk


def test_graph_survives_workspace_growth():
    import torch
    rng = rng_of(61)
    p, q = _decode(rng)
    cache, seqs = p.on_device()
    q = to_dev(q)
    big, bq = _decode(rng, sizes=((3000, 40),))
    bcache, bseqs = big.on_device()
    bq = to_dev(bq)
    want, bwant = q4k.attention(q, cache, seqs), q4k.attention(bq, bcache, bseqs)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        q4k.attention(q, cache, seqs)
        side.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            out = q4k.attention(q, cache, seqs)
        assert torch.equal(q4k.attention(bq, bcache, bseqs), bwant)
    for _ in range(3):
        out.fill_(float("nan"))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        with torch.cuda.stream(side):
            assert torch.equal(q4k.attention(bq, bcache, bseqs), bwant)
        torch.cuda.synchronize()


def test_calls_of_all_kinds_after_one_another():
    """One workspace and one set of counters: sizes, kernels and types in turn, twice, and out-of-order
    offsets in between, give each call's own result."""
    import torch
    rng = rng_of(62)
    calls = []
    for kind in ("f16", "bf16", "e4m3"):
        for sizes in (((900, 1), (40, 1)), ((700, 8),), ((10, 50), (0, 90)), ((600, 30),), tuple((b, 1) for b in range(70))):
            for D in (64, 128):
                p = Paged(rng, list(sizes), 2, D, 16, kind)
                cache, seqs = p.on_device()
                calls.append((to_dev(rng.standard_normal((p.T, 8, D)).astype(np.float32)), cache, seqs))
    first = [q4k.attention(*c) for c in calls]
    for c, want in zip(calls, first):
        assert torch.equal(q4k.attention(*c), want)
        q, cache, seqs = c
        q4k.attention(q, cache, seqs._replace(offsets=seqs.offsets.flip(0).contiguous()))
    for c, want in list(zip(calls, first))[::-1]:
        assert torch.equal(q4k.attention(*c), want)


def test_streams_and_threads_at_once():
    import torch
    rng = rng_of(63)
    work = []
    for n in range(4):
        p, q = _decode(rng, sizes=((2000 + 100 * n, 1 + 8 * n), (50, 1)))
        cache, seqs = p.on_device()
        q = to_dev(q)
        work.append((q, cache, seqs, q4k.attention(q, cache, seqs), torch.cuda.Stream()))
    torch.cuda.synchronize()
    bad = []

    def run(q, cache, seqs, want, stream):
        with torch.cuda.stream(stream):
            got = [q4k.attention(q, cache, seqs) for _ in range(30)]
            stream.synchronize()
            bad.extend(1 for g in got if not torch.equal(g, want))

    threads = [threading.Thread(target=run, args=w) for w in work]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert not bad


def _memory_stream(t):
    import torch
    at = t.data_ptr()
    for segment in torch.cuda.memory_snapshot():
        if segment["address"] <= at < segment["address"] + segment["total_size"]:
            return segment["stream"]
    raise AssertionError("not in the allocator's memory")


@pytest.mark.parametrize("handle", [False, True], ids=["stream", "handle"])
@pytest.mark.parametrize("call", ["norm", "append", "attention", "tree"])
def test_outputs_come_from_the_given_streams_memory(call, handle):
    import torch
    rng = rng_of(64)
    p, q = _decode(rng)
    cache, seqs = p.on_device()
    q, k = to_dev(q), torch.randn(3, 2, 64, device="cuda")
    x, w = torch.randn(5, 96, device="cuda"), torch.rand(96, device="cuda")
    mask = torch.ones(3, 1, dtype=torch.int32, device="cuda")
    run = {"norm": lambda st: q4k.rms_norm(x, w, residual=x, stream=st),
           "append": lambda st: q4k.kv_append(k, k, cache, seqs, q=q, stream=st),
           "attention": lambda st: q4k.attention(q, cache, seqs, stream=st),
           "tree": lambda st: q4k.attention_tree(q, cache, seqs, mask, stream=st)}[call]
    want = run(None)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = run(side.cuda_stream if handle else side)
    torch.cuda.synchronize()
    for a, b in zip(*[t if isinstance(t, tuple) else (t,) for t in (want, got)]):
        assert _memory_stream(a) == 0 and _memory_stream(b) == side.cuda_stream
        assert torch.equal(a, b)


@pytest.mark.parametrize("words", [2, 1])
@pytest.mark.parametrize("sizes", [[(40, 8), (3, 3)], [(90, 40), (20, 64)]])
def test_bits_behind_the_new_tokens_are_not_read(sizes, words):
    """Masks with every bit set beyond a sequence's own new tokens."""
    rng = rng_of(65, words)
    p = Paged(rng, sizes, 2, 64, 16, "f16")
    q = rng.standard_normal((p.T, 4, 64)).astype(np.float32)
    mask = np.full((p.T, words), 0xFFFFFFFF, np.uint32)
    cache, seqs = p.on_device()
    got = q4k.attention_tree(to_dev(q), cache, seqs, to_dev(mask.view(np.int32))).cpu().numpy()
    want, S, A = attention(p, q, 0.125, mask, words)
    assert (np.abs(got - want) <= tolerance(p, S, A, int(p.lengths.max()))).all()
