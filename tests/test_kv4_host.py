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


def test_build_without_torch():
    """libtq needs nvcc alone: without torch the build goes on, less the module that is built against it."""
    import subprocess
    import sys
    code = "import sys; sys.modules['torch'] = None\nfrom kv_cache_vector_15_b200 import build\nassert build.build_calls() is None\n"
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


def test_module_follows_torch_and_python(tmp_path, monkeypatch):
    """_calls.so is built again for another torch or interpreter, and not otherwise."""
    import types

    import torch

    from kv_cache_vector_15_b200 import build
    made = []

    def compiler(cmd, **kw):
        made.append(cmd)
        open(cmd[cmd.index("-o") + 1], "w").close()
        return types.SimpleNamespace(returncode=0)

    monkeypatch.setattr(build, "CALLS", str(tmp_path / "_calls.so"))
    monkeypatch.setattr(build, "CALLS_FOR", str(tmp_path / "calls.for"))
    monkeypatch.setattr(build.subprocess, "run", compiler)
    for count in (1, 1):
        assert build.build_calls() == build.CALLS and len(made) == count
    monkeypatch.setattr(torch, "__version__", "another")
    for count in (2, 2):
        assert build.build_calls() == build.CALLS and len(made) == count
    monkeypatch.setattr(build.sys, "version", "another")
    for count in (3, 3):
        assert build.build_calls() == build.CALLS and len(made) == count
