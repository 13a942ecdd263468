"""The work that attention over the cache lays out for its tensor-core kernel, host logic only: the
steps of 256 rows by 128 keys of a sequence, also where there are more than 32 bits count."""
import itertools

import numpy as np
import pytest


def steps(n, length, group, causal, window):
    """From the definition: row r is query r // group, which sees a range of keys; a segment of 256
    rows takes the 64-key blocks that its rows see, two a step, and at least one step."""
    p = np.arange(length - n, length)
    last = p if causal else np.where(p >= 0, length - 1, p)
    first = np.maximum(0, p - window + 1) if window > 0 else np.zeros(n, int)
    total = 0
    for r in range(0, n * group, 256):
        rows = slice(r // group, (min(r + 256, n * group) - 1) // group + 1)
        sees = last[rows] >= first[rows]
        lo, hi = (first[rows][sees].min() // 64, last[rows][sees].max() // 64 + 1) if sees.any() else (0, 0)
        total += max(1, -(-(hi - lo) // 2))
    return total


@pytest.mark.parametrize("n,length", [(0, 0), (1, 1), (1, 500), (60, 40), (300, 300), (300, 0), (700, 5000), (1000, 999)])
def test_steps_of_small_sequences(libsa, n, length):
    f = libsa.raw_library().sa_debug_cache_steps
    for group, causal, window in itertools.product((1, 3, 8, 300), (0, 1), (0, 1, 64, 200, 1 << 30)):
        assert f(n, length, group, causal, window) == steps(n, length, group, causal, window), (group, causal, window)


@pytest.mark.parametrize("n,group", [(2_000_000, 40), (1 << 23, 8), (1 << 30, 1), (1 << 21, 512)])
def test_steps_past_32_bits(libsa, n, group):
    """All the segments of a sequence of n tokens: without causality each takes every block."""
    f = libsa.raw_library().sa_debug_cache_steps
    want = -(-n * group // 256) * -(-(-(-n // 64)) // 2)
    assert f(n, n, group, 0, 0) == want and want > 1 << 31
    assert want // 2 < f(n, n, group, 1, 0) < want // 2 + want // 1000


def test_refused_sizes(libsa):
    f = libsa.raw_library().sa_debug_cache_steps
    assert f(-1, 1, 1, 0, 0) == f(1, -1, 1, 0, 0) == f(1, 1, 0, 0, 0) == f(1, 1, 1, 0, -1) == -1
    assert f(1, (1 << 30) + 1, 1, 0, 0) == f(1 << 20, 1, 1 << 11, 0, 0) == -1
