"""Pins of oracle/kv4.py on the CPU at the ends of what the 4-bit form holds."""

import numpy as np

from oracle import kv4 as o


def test_a_nan_makes_its_group_nan():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((4, 192)).astype(np.float32)
    plain = o.quantize(x)
    x[1, 70], x[2, 128:], x[3, [0, 1]] = np.nan, np.nan, (np.inf, np.nan)
    bad = np.isnan(x).reshape(4, 3, 64).any(-1)
    c, s, z = o.quantize(x)
    assert np.array_equal(np.isnan(o.values(c, s, z)), np.repeat(bad, 64, -1))
    assert np.all(s.view(np.uint16)[bad] == 0x7fff) and np.all(z.view(np.uint16)[bad] == 0x7fff) and not c[np.repeat(bad, 64, -1)].any()
    for a, b in zip((s, z), plain[1:]):
        assert np.array_equal(a[~bad], b[~bad])
    assert np.array_equal(c[~np.repeat(bad, 64, -1)], plain[0][~np.repeat(bad, 64, -1)])


def test_codes_are_those_of_the_exact_quotient():
    """Against rational numbers: random groups, and coordinates on and next to
    the borders between codes, some nearer than 64 bits show in x - z."""
    from fractions import Fraction
    rng = np.random.default_rng(1)
    x = (rng.standard_normal((60, 64)) * np.exp(3 * rng.standard_normal((60, 1)))).astype(np.float32)
    for i in range(20):
        s, k = np.float32(2.0 ** (i % 5 - 2)), i % 15
        z = -np.float32(k + 0.5) * s                             # zero is the border behind code k
        x[i] = np.resize(np.float32([z, z + 15 * s, 0.0, 1e-30, -1e-30, 2.0 ** -149, -(2.0 ** -60), s, -s, 0.5 * s]), 64)
        x[i] = np.clip(x[i], z, z + 15 * s)
    c, s, z = o.quantize(x)
    for i in range(60):
        S, Z = Fraction(float(s[i, 0])), Fraction(float(z[i, 0]))
        want = [min(max(round((Fraction(float(v)) - Z) / S), 0), 15) if S else 0 for v in x[i]]   # ties to the even one
        assert c[i].tolist() == want, i
