"""The search for a token's sequence (q4k_cache.h), its steps written out: every token of ascending
offsets finds its own sequence, and offsets out of order stay in range."""
import numpy as np
import pytest


def last_started(start, at):
    """A wave's search: 64 lanes, each step keeps a 64th of the range."""
    low, span = 0, len(start)
    lanes = np.arange(64)
    while span > 64:
        step = (span + 63) // 64
        i = lanes * step
        begun = (i < span) & (start[np.minimum(low + i, len(start) - 1)] <= at)
        more = max(int(begun.sum()) - 1, 0) * step
        low += more
        span = min(step, span - more)
    begun = (lanes < span) & (start[np.minimum(low + lanes, len(start) - 1)] <= at)
    return low + max(int(begun.sum()) - 1, 0)


@pytest.mark.parametrize("count", [1, 2, 63, 64, 65, 127, 128, 129, 4095, 4096, 4097, 5000, 65535])
def test_every_token_finds_its_sequence(count):
    rng = np.random.Generator(np.random.PCG64(count))
    n = rng.integers(0, 3, count) * (rng.random(count) < 0.7)
    n[0] = rng.integers(0, 2)
    offsets = np.concatenate([[0], np.cumsum(n)])
    total = int(offsets[-1])
    for t in {0, 1, total // 2, total - 1, *rng.integers(0, max(total, 1), 200).tolist()}:
        if not 0 <= t < total:
            continue
        b = last_started(offsets[:-1], t)
        assert offsets[b] <= t < offsets[b + 1]


def test_offsets_out_of_order_stay_in_range():
    rng = np.random.Generator(np.random.PCG64(7))
    for count in (1, 3, 64, 65, 200, 4500):
        for _ in range(50):
            offsets = rng.integers(0, 1000, count)
            assert 0 <= last_started(offsets, int(rng.integers(0, 1000))) < count
