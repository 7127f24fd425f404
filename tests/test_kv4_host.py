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


def test_lists_of_slots_that_32_bits_do_not_count(tq):
    """The new tokens' places in the list are 32-bit numbers: longer lists are refused."""
    before = tq.launch_count()
    at = 1 << 20                                                 # addresses that nothing reads
    t = tq._Pages(at, at + 4096, at + 8192, 6, 5, 20, 16, 0)
    for n_slots in (1 << 31, 1 << 40):
        assert tq.call_status("tq_pages_extend", t, t, 1, at, at, at, n_slots, at, 1 << 20, 0) == tq.TQ_ERR_INVALID_ARG
        assert "n_slots" in tq.last_error()
    assert tq.launch_count() == before
