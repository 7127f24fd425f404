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
