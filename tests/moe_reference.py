"""Plain 64-bit forms of the mixture-of-experts operators, for the tests.

Independent of the library and of the C oracle: Q4_K blocks are unpacked from
the format's description with numpy, and every product is a float64 product.
"""
from __future__ import annotations

import numpy as np


def unpack(w):
    """(weights, magnitudes) float64 [N, K] of packed rows [N, K/256*144]: w = d*sc*q
    - dmin*m and |d|*sc*q + |dmin|*m, the sum of its two terms' magnitudes."""
    N = w.shape[0]
    b = np.ascontiguousarray(w).reshape(-1, 144)
    d = b[:, 0:2].copy().view(np.float16).astype(np.float64)
    dmin = b[:, 2:4].copy().view(np.float16).astype(np.float64)
    s = b[:, 4:16].astype(np.int64)
    val = np.empty((b.shape[0], 8, 32))
    mag = np.empty_like(val)
    for j in range(8):
        if j < 4:
            sc, m = s[:, j] & 63, s[:, j + 4] & 63
        else:
            sc = (s[:, j + 4] & 15) | ((s[:, j - 4] >> 6) << 4)
            m = (s[:, j + 4] >> 4) | ((s[:, j] >> 6) << 4)
        raw = b[:, 16 + 32 * (j // 2):48 + 32 * (j // 2)]
        q = (raw >> 4 if j % 2 else raw & 15).astype(np.float64)
        val[:, j] = d * sc[:, None] * q - dmin * m[:, None]
        mag[:, j] = np.abs(d) * sc[:, None] * q + np.abs(dmin) * m[:, None]
    return val.reshape(N, -1), mag.reshape(N, -1)


def grouped(w, x, offsets, rows, x_div, P):
    """(y, s) float64 [P, N]: the grouped products and sum_k |x_k| * magnitude_k;
    NaN in rows of pairs that no group names."""
    E, N = w.shape[0], w.shape[1]
    y = np.full((P, N), np.nan)
    s = np.full((P, N), np.nan)
    x = x.astype(np.float64)
    for e in range(E):
        r = np.asarray(rows[offsets[e]:offsets[e + 1]])
        r = r[(r >= 0) & (r < P)]
        if len(r) == 0:
            continue
        val, mag = unpack(w[e])
        y[r] = x[r // x_div] @ val.T
        s[r] = np.abs(x[r // x_div]) @ mag.T
    return y, s


def product_tol(K):
    """Relative to s: x as hi + lo binary16 is off by at most 2^-22 of each value
    (two roundings of 2^-11); a sum of 2K products and 2K/256 scalings in fp32,
    each rounding at most 2^-24 of the running sum, grows like a random walk:
    four standard deviations of sqrt(2K) of them."""
    return 2.0 ** -22 + 4.0 * np.sqrt(2.0 * K) * 2.0 ** -24


def silu(z):
    with np.errstate(over="ignore"):
        return z / (1.0 + np.exp(-z))


def stable_groups(expert, E):
    """(offsets, rows) of a flat table of choices; the tail of rows is -1."""
    flat = np.asarray(expert).reshape(-1).astype(np.int64)
    ok = (flat >= 0) & (flat < E)
    order = np.argsort(np.where(ok, flat, E), kind="stable")
    offsets = np.concatenate([[0], np.cumsum(np.bincount(flat[ok], minlength=E)[:E])]).astype(np.int32)
    rows = np.where(np.arange(flat.size) < offsets[-1], order, -1).astype(np.int32)
    return offsets, rows


def route(logits, bias, top_k, sigmoid, normalize, scale):
    """(expert, weight) by the definition in float64."""
    z = logits.astype(np.float64)
    ok = z > -np.inf  # false for NaN
    zz = np.where(ok, z, -np.inf)
    with np.errstate(over="ignore", invalid="ignore"):
        if sigmoid:
            score = np.where(ok, 1.0 / (1.0 + np.exp(-zz)), 0.0)
        else:
            mx = zz.max(axis=1, keepdims=True)
            term = np.where(zz == mx, 1.0, np.exp(zz - mx)) * ok
            total = term.sum(axis=1, keepdims=True)
            score = term / np.where(total > 0, total, 1.0)
    # without a bias the logits decide (the same order, no rounding between)
    by = zz if bias is None else np.where(ok, score + bias.astype(np.float64), -np.inf)
    by = np.where(np.isnan(by), -np.inf, by)
    order = np.argsort(-by, axis=1, kind="stable")[:, :top_k]
    chosen = np.take_along_axis(by, order, 1) > -np.inf
    expert = np.where(chosen, order, -1).astype(np.int32)
    weight = np.where(chosen, np.take_along_axis(score, order, 1), 0.0)
    if normalize:
        total = weight.sum(axis=1, keepdims=True)
        weight = np.where(total > 0, weight / np.where(total > 0, total, 1.0), 0.0)
    return expert, scale * weight
