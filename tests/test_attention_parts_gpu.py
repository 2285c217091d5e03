"""A bfloat16 cache's products go by three bfloat16 parts of every query and weight: inputs
at which two parts (or a part forgotten) would be far outside what is granted, through
the tiles of 16, 32, 64 and 128 rows.  The same inputs through a form with two parts on
the CPU show that these tests would see it."""
import numpy as np
import pytest

import gguf_q4_dequant_amd as q4k
from tests.gpu_helpers import to_dev
from tests.layer_reference import Paged, rng_of

D, HQ, HK, PAGE = 64, 8, 2, 16
SCORE = 100.0  # the scores' size in the test of the queries

# New tokens behind a context: four query heads a key head make rows for the tiles of 16, 32, 64 and 128.
SIZES = {"16 rows": [(300, 1), (90, 2)], "32 rows": [(300, 8)], "64 rows": [(300, 16)], "128 rows": [(300, 40)],
         "prompt": [(0, 90)], "many tiles": [(9 * b % 70, 1) for b in range(130)]}


def to_bf16(x):
    """float32 values (as float64) to the nearest bfloat16, ties to even."""
    u = np.asarray(x, np.float32).view(np.uint32).astype(np.uint64)
    u = (u + 0x7FFF + (u >> 16 & 1)) & 0xFFFF0000
    return u.astype(np.uint32).view(np.float32).astype(np.float64)


def in_parts(x, parts):
    """x as the sum of its bfloat16 parts."""
    rest, total = np.asarray(x, np.float32).astype(np.float64), 0.0
    for _ in range(parts):
        h = to_bf16(rest)
        total, rest = total + h, rest - h
    return total


def queries_case(rng, rows):
    """q [rows, 2], near SCORE / (scale * key) each: keys of dimension 0 have value 1, those of dimension 1
    have -1.  Rows' scores differ by 2 at most, so that out = tanh of half the difference is not flat."""
    x = 1 + rng.random(rows)
    return np.stack([x, x * (1 + (rng.random(rows) - 0.5) * 2 / SCORE / 2)], 1).astype(np.float32)


def plain_queries(q, key, scale, parts, first, second):
    """The output over `first` keys of dimension 0 and `second` of dimension 1, per row."""
    split = in_parts(q, parts) if parts else q.astype(np.float64)
    s = scale * key * split
    d = s[:, 0] - s[:, 1]
    return (first * np.exp(d) - second) / (first * np.exp(d) + second)


# Scores: x * by, two additions of parts and the rounding of the product's operand are 2^-24 of SCORE * 2
# each (x is up to 2), of two scores; out moves by half of their difference.  The exponent's argument (up
# to 16 and a shift) is good to 2^-20 and the exponential to 2^-22, the sums of up to 340 equal weights to
# 4 * sqrt(340) * 2^-24; twice that covers numerator and denominator.
QUERY_TOL = 0.5 * 8 * 2.0 ** -24 * 2 * SCORE + 2 * (2.0 ** -20 + 2.0 ** -22 + 4 * 340 ** 0.5 * 2.0 ** -24)


def test_two_parts_of_the_queries_would_be_seen():
    rng = rng_of(70)
    q = queries_case(rng, 64)
    key, scale = 32.0, SCORE / 32
    want = plain_queries(q, key, scale, 0, 5, 5)
    assert np.abs(plain_queries(q, key, scale, 3, 5, 5) - want).max() <= QUERY_TOL / 4
    assert np.abs(plain_queries(q, key, scale, 2, 5, 5) - want).max() >= 4 * QUERY_TOL


def filled(sizes, **more):
    """Paged sequences in bfloat16 of which every place that they have holds zeros."""
    p = Paged(rng_of(71), sizes, HK, D, PAGE, "bf16", **more)
    for b in range(len(sizes)):
        for j in range(int(p.lengths[b])):
            at = int(p.table[b, j // PAGE]), slice(None), j % PAGE
            p.k[at], p.v[at] = 0, 0
    return p


def set_place(p, b, j, dim, key, value):
    at = int(p.table[b, j // PAGE]), slice(None), j % PAGE
    p.k[(*at, dim)] = key
    p.v[at] = value


@pytest.mark.gpu
@pytest.mark.parametrize("name", SIZES)
def test_queries_of_every_kernel(name):
    sizes = SIZES[name]
    rng = rng_of(72, list(SIZES).index(name))
    p = filled(sizes, extra_cols=400)
    key, scale = 32.0, SCORE / 32
    for b in range(len(sizes)):
        for j in range(int(p.lengths[b])):
            set_place(p, b, j, j % 2, key, 1 - 2 * (j % 2))
    T = p.T
    pair = queries_case(rng, T * HQ)
    q = np.zeros((T, HQ, D), np.float32)
    q[..., :2] = pair.reshape(T, HQ, 2)
    cache, seqs = p.on_device()
    got = q4k.attention(to_dev(q), cache, seqs, scale).cpu().numpy()
    for b in range(len(sizes)):
        for t in range(int(p.offsets[b]), int(p.offsets[b + 1])):
            keys = int(p.lengths[b]) - int(p.offsets[b + 1]) + t + 1
            want = plain_queries(q[t, :, :2], key, np.float32(scale).astype(np.float64), 0, (keys + 1) // 2, keys // 2)
            assert (np.abs(got[t] - want[:, None]) <= QUERY_TOL).all(), (t, np.abs(got[t] - want[:, None]).max())


def plain_weights(x, parts):
    """w2 / (w1 + w2) of scores x and 0 (x in [0.25, 4]), the numerator's weight in parts."""
    w = np.exp(-x.astype(np.float64))
    return (in_parts(w, parts) if parts else w) / (1 + w)


# Relative: three roundings of x and one of the argument's sum (|argument| < 32) move the exponent by
# 4 * 2^-24 * 4 + 2^-20 at most, times ln 2 for the last; the exponential, the parts, the sum, the quotient
# and the product add 2^-22 + 4 * 2^-24.
WEIGHT_TOL = 4 * 2.0 ** -24 * 4 + 2.0 ** -20 * 0.6932 + 2.0 ** -22 + 4 * 2.0 ** -24


def test_two_parts_of_the_weights_would_be_seen():
    x = (0.25 + 3.75 * rng_of(73).random(512)).astype(np.float32)
    want = plain_weights(x, 0)
    assert (np.abs(plain_weights(x, 3) - want) <= WEIGHT_TOL / 4 * want).all()
    assert (np.abs(plain_weights(x, 2) - want) / want).max() >= 2 * WEIGHT_TOL


@pytest.mark.gpu
@pytest.mark.parametrize("name", SIZES)
def test_weights_of_every_kernel(name):
    """The first key of a sequence has the largest score and a value of zero, its second key a score of 0 and
    a value of one; the keys behind have scores whose weights are nothing."""
    sizes = SIZES[name]
    rng = rng_of(74, list(SIZES).index(name))
    p = filled(sizes, extra_cols=400)
    for b in range(len(sizes)):
        for j in range(int(p.lengths[b])):
            at = int(p.table[b, j // PAGE]), slice(None), j % PAGE
            p.k[(*at, 0)], p.k[(*at, 1)] = float(j == 0), -1000.0 * (j > 1)
            p.v[at] = float(j == 1)
    T = p.T
    x = (0.25 + 3.75 * rng.random((T, HQ))).astype(np.float32)
    q = np.zeros((T, HQ, D), np.float32)
    q[..., 0], q[..., 1] = x, 1
    cache, seqs = p.on_device()
    got = q4k.attention(to_dev(q), cache, seqs, 1.0).cpu().numpy()
    for b in range(len(sizes)):
        for t in range(int(p.offsets[b]), int(p.offsets[b + 1])):
            if int(p.lengths[b]) - int(p.offsets[b + 1]) + t == 0:
                assert (got[t] == 0).all()  # only the first key
                continue
            want = plain_weights(x[t], 0)[:, None]
            assert (np.abs(got[t] - want) <= WEIGHT_TOL * want).all(), (t, (np.abs(got[t] - want) / want).max())
