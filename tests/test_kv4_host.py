"""Host-side behaviour of the paged 4-bit cache's binding and its build.  Needs no GPU."""

import numpy as np
import pytest


@pytest.fixture(scope="module")
def tq():
    from kv_cache_vector_15_b200 import tq as _tq
    return _tq


def test_rope_plans_hold_their_own_numbers(tq):
    """The kernels read a plan by its arrays' addresses: those cannot be replaced, and the caller's arrays are not shared."""
    inv, axis = np.ones(8), np.zeros(8, np.int32)
    p = tq.Rope(inv, axis=axis)
    inv[:] = 7.0
    axis[:] = 3
    assert np.all(p.inv_freq == 1.0) and np.all(p.axis == 0)
    assert p._c[2:] == (p.inv_freq.ctypes.data, p.axis.ctypes.data)
    for name in ("inv_freq", "axis", "interleaved", "rot_dim"):
        with pytest.raises(AttributeError):
            setattr(p, name, getattr(p, name))
    wide = np.arange(32.0).reshape(16, 2)[::-1, 0]
    assert tq.Rope(wide).inv_freq.flags.c_contiguous and np.array_equal(tq.Rope(wide).inv_freq, wide)
