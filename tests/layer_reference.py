"""Plain float64 forms of the operators of include/q4k_layer.h, one sequence and
head at a time, and the paged inputs of their tests."""
import math

import numpy as np

import q4k_inputs as qi

TYPES = ("f16", "bf16", "e4m3")


def rng_of(*path):
    return np.random.Generator(np.random.PCG64(qi.tensor_seed(qi.BASE_SEED, 1500, *path)))


def torch_type(name):
    import torch
    return {"f16": torch.float16, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}[name]


def rounded(a, name):
    """a rounded to the type (e4m3 saturating), as a torch tensor of it on the CPU."""
    import torch
    t = torch.from_numpy(np.ascontiguousarray(a, dtype=np.float64))
    if name == "e4m3":
        t = t.clamp(-448, 448)
    return t.to(torch_type(name))


class Paged:
    """Sequences of (context, new tokens) in a paged pool; every place that no
    sequence has holds NaN, infinities or the type's largest values."""

    def __init__(self, rng, sizes, kv_heads, D, page, kind, k_scale=1.0, v_scale=1.0, spare=3, extra_rows=0, extra_cols=0,
                 new_empty=False):
        import torch
        self.sizes, self.kv_heads, self.D, self.page, self.kind = sizes, kv_heads, D, page, kind
        self.k_scale, self.v_scale = k_scale, v_scale
        n = [m for _, m in sizes]
        self.lengths = np.array([c + m for c, m in sizes], np.int32)
        self.offsets = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
        self.T = int(self.offsets[-1]) + extra_rows
        need = [max(0, -(-int(l) // page)) for l in self.lengths]
        self.pool = sum(need) + spare
        order = rng.permutation(self.pool)
        self.table = np.full((len(sizes), max(need + [0]) + extra_cols), -1, np.int32)
        at = 0
        for b, k in enumerate(need):
            self.table[b, :k] = order[at:at + k]
            at += k
        shape = (self.pool, kv_heads, page, D)
        junk = np.array([np.nan, np.inf, -np.inf, 448.0, -448.0])
        k, v = rng.choice(junk, shape), rng.choice(junk, shape)
        for b, (c, m) in enumerate(sizes):
            for j in range(max(c, 0) if new_empty else max(c + m, 0)):
                p = self.table[b, j // page]
                k[p, :, j % page] = (rng.standard_normal((kv_heads, D)) + 0.5) / k_scale
                v[p, :, j % page] = rng.standard_normal((kv_heads, D)) / v_scale
        if kind == "e4m3":  # no infinities there
            k, v = np.where(np.isinf(k), np.nan, k), np.where(np.isinf(v), np.nan, v)
        self.k, self.v = rounded(k, kind), rounded(v, kind)
        self.torch = torch

    def on_device(self):
        """(KVCache, Sequences) on the GPU."""
        import gguf_q4_dequant_amd as q4k
        t = lambda a: self.torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
        return (q4k.KVCache(self.k.cuda(), self.v.cuda(), self.k_scale, self.v_scale),
                q4k.Sequences(t(self.offsets), t(self.lengths), t(self.table)))

    def values(self, k=None, v=None):
        """The cache's values in 64 bits."""
        k, v = self.k if k is None else k, self.v if v is None else v
        return k.double().numpy() * self.k_scale, v.double().numpy() * self.v_scale


def attention(p, q, scale, mask=None, words=0):
    """(out, S, A) in 64 bits: S[0] = sum_j p_j |v_j|; S[1] = sum_j |v_j| over the
    sum of the weights relative to the largest one (what the smallest weights'
    rounding goes by); A [T, Hq] = the largest scale * sum_d |q_d k_jd| of a row (what
    the scores' rounding goes by)."""
    k, v = p.values()
    T, Hq, D = q.shape
    G = Hq // p.kv_heads
    q = q.astype(np.float64)
    out, S, A = np.zeros(q.shape), np.zeros((2, *q.shape)), np.zeros((T, Hq))
    for b in range(len(p.sizes)):
        first, end, L = int(p.offsets[b]), int(p.offsets[b + 1]), int(p.lengths[b])
        n = end - first
        idx = np.arange(max(L, 0))
        col = idx // p.page
        ok = col < p.table.shape[1]
        page = np.where(ok, p.table[b][np.minimum(col, max(p.table.shape[1] - 1, 0))] if p.table.shape[1] else -1, -1)
        idx, page = idx[(page >= 0) & (page < p.pool)], page[(page >= 0) & (page < p.pool)]
        if not len(idx):
            continue
        for i in range(n):
            t = first + i
            if mask is None:
                see = idx <= L - n + i
            else:
                new = idx - (L - n)
                word = mask[t][np.clip(new >> 5, 0, words - 1)].astype(np.int64) & 0xFFFFFFFF
                see = (new < 0) | ((new < 32 * words) & ((word >> (new & 31)) & 1 != 0))
            if not see.any():
                continue
            for h in range(Hq):
                kk, vv = k[page[see], h // G, idx[see] % p.page], v[page[see], h // G, idx[see] % p.page]
                with np.errstate(invalid="ignore", over="ignore"):
                    s = scale * (kk @ q[t, h])
                    top = s.max()
                    if top == -math.inf:
                        continue
                    e = np.exp(s - top)
                    w = e / e.sum()
                    out[t, h] = w @ vv
                    S[0, t, h] = w @ np.abs(vv)
                    S[1, t, h] = np.abs(vv).sum(0) / e.sum()
                    A[t, h] = abs(scale) * (np.abs(kk) @ np.abs(q[t, h])).max()
    return out, S, A


def tolerance(p, S, A, longest):
    """What out may be off, elementwise.  A score is off by the split of q (2^-21 of each
    product at most; 2^-16 are granted over a bfloat16 cache) and by the sum of D float32
    products (sqrt(D) roundings of 2^-24 at work, times 4), relative to A; the exponent's
    argument and the hardware's exponential add |s| 2^-23 and 2^-22; numerator and
    denominator each carry it (times 2), the weights' split adds as much as q's, and
    the sum over the keys sqrt(keys) roundings (times 4).  A weight is held with an
    absolute error beside the relative one: binary16's subnormal numbers end at
    2^-24, half a step is 2^-25, and the largest weight is held as 2^13 or more, which
    makes 2^-38 of it (float32's own end, 2^-150, is far below)."""
    split = 2.0 ** -16 if p.kind == "bf16" else 2.0 ** -21
    score = (split + 4 * math.sqrt(p.D) * 2.0 ** -24 + 2.0 ** -23) * A[:, :, None]
    return (2 * (score + 2.0 ** -22) + split + 4 * math.sqrt(max(longest, 1)) * 2.0 ** -24) * S[0] + 2.0 ** -38 * S[1]


def rotation(x, weight, eps, positions, inv_freq, interleaved):
    """x [T, H, D] normed (weight, or None) and rotated, and the size of each value's pair, in 64 bits."""
    x = x.astype(np.float64)
    if weight is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * weight.astype(np.float64)
    y, size = x.copy(), np.abs(x)
    if inv_freq is not None and len(inv_freq):
        R = 2 * len(inv_freq)
        angle = positions.astype(np.float64)[:, None] * inv_freq.astype(np.float64)[None]
        c, s = np.cos(angle)[:, None], np.sin(angle)[:, None]
        at = (slice(0, R, 2), slice(1, R, 2)) if interleaved else (slice(0, R // 2), slice(R // 2, R))
        a, b = x[..., at[0]], x[..., at[1]]
        y[..., at[0]], y[..., at[1]] = a * c - b * s, b * c + a * s
        size[..., at[0]] = size[..., at[1]] = np.hypot(a, b)
    return y, size


def tree_mask(rng, sizes, words, extra_rows=0):
    """uint32 masks [T, words] of random trees: a token sees itself and the tokens that it follows."""
    rows = []
    for _, n in sizes:
        seen = []
        for i in range(n):
            up = int(rng.integers(-1, i)) if i else -1
            seen.append((seen[up] if up >= 0 else 0) | 1 << i)
            rows.append([seen[i] >> 32 * w & 0xFFFFFFFF for w in range(words)])
    rows += [[0] * words] * extra_rows
    return np.array(rows, np.uint32).reshape(-1, words)
