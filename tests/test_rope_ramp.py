"""The ramp of rotation frequencies where its borders lie outside the pairs: contexts so long that
every pair turns more than beta_slow times, and so short that every pair turns less."""
import math

import numpy as np
import pytest


def ramp(rot, base, factor, length, fast, slow):
    """(share of the slowed frequency, turns within length) of each pair, from the definition: the
    index at which a pair would turn fast (slow) times, rounded down (up), begins (ends) the mix."""
    i = np.arange(rot // 2)
    turns = length * base ** (-2.0 * i / rot) / (2 * math.pi)
    first, last = (rot / 2 * math.log(length / (2 * math.pi * t)) / math.log(base) for t in (fast, slow))
    lo, hi = math.floor(first), math.ceil(last)
    return np.clip((i - lo) / (hi - lo), 0.0, 1.0), turns


@pytest.mark.parametrize("rot,base,factor,length,fast,slow", [
    (128, 10000.0, 4.0, 65536, 32.0, 1.0), (128, 10000.0, 4.0, 131072, 32.0, 1.0), (128, 10000.0, 8.0, 1 << 20, 32.0, 1.0),
    (64, 10000.0, 4.0, 1 << 20, 32.0, 1.0), (16, 10000.0, 4.0, 65536, 32.0, 1.0), (16, 10000.0, 4.0, 4, 32.0, 1.0),
    (128, 10000.0, 4.0, 6, 32.0, 1.0), (128, 10000.0, 4.0, 1, 32.0, 1.0), (128, 500000.0, 32.0, 8192, 32.0, 1.0),
    (32, 2.0, 4.0, 100, 1000.0, 100.0), (32, 2.0, 4.0, 100, 1.0, 0.5), (96, 10000.0, 2.0, 4096, 4096.0, 1e-3),
])
def test_ramp_follows_its_formula(libsa, rot, base, factor, length, fast, slow):
    share, turns = ramp(rot, base, factor, length, fast, slow)
    plain = base ** (-2.0 * np.arange(rot // 2) / rot)
    f, a = libsa.sa_rope_frequencies(rot, base, "ramp", factor, length, fast, slow, device="cpu")
    # a handful of roundings in 64 bits, logarithms of up to 20 times the result among them
    assert np.allclose(f.numpy(), plain * (1.0 - share) + plain / factor * share, rtol=1e-12, atol=0)
    assert math.isclose(a, 0.1 * math.log(factor) + 1, rel_tol=1e-6)
    got = (plain - f.numpy()) / (plain - plain / factor)
    assert np.all(got[turns <= slow] >= 1 - 1e-12), "a pair below beta_slow keeps some of its frequency"
    assert np.all(np.abs(got[turns >= fast]) <= 1e-12), "a pair above beta_fast is slowed"
    inside = (turns > slow * base ** (2 / rot)) & (turns < fast / base ** (2 / rot))
    assert np.all(got[inside] < 1) and np.all(got[inside] > 0), "a pair between the borders is not mixed"
