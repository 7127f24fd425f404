"""Calls of the page table that have to be refused, or done whole: bad entries in
rows, no room for slots, tables of another device, layouts that read two ways."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]


@pytest.fixture(scope="module")
def tq():
    from kv_cache_vector_15_b200 import tq as _tq
    return _tq


def i32(x):
    return torch.tensor(list(x), dtype=torch.int32, device="cuda")


def arrays(T):
    return [x.clone() for x in (T.table, T.lens, T.refs)]


def other(tq, T):
    return tq.PageTable(torch.full_like(T.table, 77), torch.full_like(T.lens, 78), torch.full_like(T.refs, 79), T.page_size)


def unchanged(tq, T, before, out, call):
    """The call is recorded as a bad one and leaves in's contents in out."""
    r = call()
    with pytest.raises(tq.TQError) as e:
        T.check()
    assert e.value.status == tq.TQ_ERR_INVALID_ARG
    assert all(torch.equal(x, y) for x, y in zip(before, arrays(T)))
    if out is not None:
        assert all(torch.equal(x, y) for x, y in zip(before, arrays(out)))
    return r


@pytest.mark.parametrize("n,m", [(8, 4), (5, 9)])
def test_pools_that_read_two_ways(tq, n, m):
    """[n, n, m] is one layer of n pages or n layers of n pages: the call asks which."""
    pool = torch.arange(n * n * m, device="cuda", dtype=torch.int32).view(n, n, m)
    pairs = i32([1, 0, 2, n - 1, -1, -1]).view(3, 2)
    keep = pool.clone()
    with pytest.raises(ValueError, match="n_layers"):
        tq.copy_pages(pool, pairs, n)
    with pytest.raises(ValueError, match="n_layers"):
        tq.PageMoves(pairs, n).copy(pool)
    assert torch.equal(pool, keep)
    one, all_of = keep.clone(), keep.clone()
    one[0], one[n - 1] = keep[1], keep[2]
    all_of[:, 0], all_of[:, n - 1] = keep[:, 1], keep[:, 2]
    a, b = pool.clone(), pool.clone()
    tq.copy_pages(a, pairs, n, n_layers=1)
    tq.PageMoves(pairs, n).copy(b, n_layers=n)
    assert torch.equal(a, one) and torch.equal(b, all_of)
    tq.copy_pages(a.view(1, n, n, m), pairs, n)                  # one reading: layers first
    tq.copy_pages(b[0], pairs, n)
    tq.copy_pages(pool.view(n, n * m), pairs, n)
    assert torch.equal(pool, one)
    with pytest.raises(ValueError):
        tq.copy_pages(pool, pairs, n, n_layers=2)
    with pytest.raises(ValueError):
        tq.copy_pages(pool, pairs, n + 1, n_layers=1)
    with pytest.raises(ValueError):
        tq.copy_pages(pool.view(n * n, m), pairs, n, n_layers=n)
    tq.copy_pages(torch.zeros((1, 1, 4), device="cuda"), i32([0, 0]).view(1, 2), 1)      # one page: both readings are one
    with pytest.raises(ValueError):
        tq.copy_pages(pool, pairs, n, n_layers=0)


def test_no_room_for_slots_is_no_room(tq):
    """n_slots = 0 is a list of no slots, not a call without a list."""
    T = tq.PageTable.empty(4, 4, 10, 16)
    T.extend(i32([0]), i32([20]), 20)
    T.check()
    before = arrays(T)
    s = unchanged(tq, T, before, None, lambda: T.extend(i32([3]), i32([5]), 0))
    assert s.shape == (0,) and s.dtype == torch.int64
    unchanged(tq, T, before, None, lambda: T.extend(i32([3, 0]), i32([0, 1]), 0))
    T.extend(i32([3, 0]), i32([0, 0]), 0)
    T.check()


@pytest.mark.parametrize("into", [False, True])
@pytest.mark.parametrize("at,entry", [(0, -1), (0, 12), (1, 1 << 30), (0, "free"), (2, -7), (2, 12), (2, "free")])
def test_bad_entries_leave_all_as_it_was(tq, into, at, entry):
    """A row whose entry is no page, or a page that nobody owns: none of the
    calls that go by the row does part of its work."""
    T = tq.PageTable.empty(6, 4, 12, 16)
    T.extend(i32([1, 0, 2, 4]), i32([30, 40, 17, 5]), 92)        # row 0: two full pages and a tail
    T.free(i32([1]))                                             # a hole, so that compaction moves
    T.check()
    T.table[0, at] = int(torch.nonzero(T.refs == 0)[-1]) if entry == "free" else entry
    before = arrays(T)
    out = other(tq, T) if into else None
    m = unchanged(tq, T, before, out, lambda: T.fork(i32([2, 0]), i32([3, 5]), out=out))
    assert torch.all(m.pairs == -1)
    unchanged(tq, T, before, out, lambda: T.free(i32([2, 0, 2]), out=out))
    m = unchanged(tq, T, before, out, lambda: T.compact(out=out))
    assert torch.all(m.pairs == -1)
    # calls that do not go by the row are done
    m = T.fork(i32([2]), i32([3]), out=out)
    T.check()
    assert (out or T).lens.tolist() == [40, 0, 17, 17, 5, 0] and int((m.pairs >= 0).sum()) == 2


def test_bad_entries_of_many_rows(tq):
    """One bad entry in a table of rows for many CTAs, whichever row has it."""
    n = 9000
    T = tq.PageTable.empty(n, 3, 3 * n, 16)
    T.extend(i32(range(n)), i32([33] * n), 33 * n)
    T.check()
    for row in (0, 31, 4567, n - 1):
        T.table[row, 1] = -3
        before = arrays(T)
        unchanged(tq, T, before, None, lambda: T.free(i32(range(n))))
        unchanged(tq, T, before, None, lambda: T.compact())
        T.table[row, 1] = before[0][row, 0] + 1
    T.free(i32(range(n)))
    T.check()
    assert not T.refs.any() and torch.all(T.table == -1)


def test_tables_of_another_device(tq):
    """Where out's arrays are is checked as in's are (here: on the host; the addresses are T's own)."""
    T = tq.PageTable.empty(4, 4, 10, 16)
    T.extend(i32([0]), i32([20]), 20)
    T.check()
    before, launches = arrays(T), tq.launch_count()

    class Far:
        table, _at = T.table.cpu(), T._at

    for call in (lambda: T.extend(i32([0]), i32([1]), 1, out=Far), lambda: T.fork(i32([0]), i32([1]), out=Far),
                 lambda: T.free(i32([0]), out=Far), lambda: T.compact(out=Far)):
        with pytest.raises(ValueError, match="cpu"):
            call()
    assert tq.launch_count() == launches
    assert all(torch.equal(x, y) for x, y in zip(before, arrays(T)))


def test_arrays_cannot_be_replaced(tq):
    """A table or cache holds its arrays' addresses: others cannot be put in their place."""
    T, C = tq.PageTable.empty(2, 2, 4, 16), tq.KV4Cache.empty(2, 1, 64, 16)
    for x, names in ((T, ("table", "lens", "refs", "status", "page_size", "n_pages")),
                     (C, ("pool", "status", "kv_heads", "d", "page_size"))):
        for name in names:
            with pytest.raises(AttributeError):
                setattr(x, name, getattr(x, name))


def test_outputs_of_dequant_on_another_stream(tq):
    """What a call on a given stream returns may go while the calling stream still reads it."""
    C = tq.KV4Cache.empty(64, 8, 128, 16)
    x = torch.randn((1024, 8, 128), device="cuda")
    slots = torch.arange(1024, device="cuda")
    C.append(x, x, slots)
    want = C.dequant(slots)[0]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    k, v = C.dequant(slots, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(100_000_000)
    got = k.clone()                                              # behind the pause
    del k, v
    with torch.cuda.stream(side):
        junk = [torch.full_like(want, float("nan")) for _ in range(4)]
    torch.cuda.synchronize()
    assert torch.equal(got, want) and len(junk) == 4


def test_errors_of_the_runtime_do_not_stay(tq):
    """A call that the CUDA runtime refuses reports it, and the thread's last
    error is not left to whoever asks next.  (The status call waits for its
    stream, which a stream under capture does not allow.)"""
    import ctypes
    rt = ctypes.CDLL("libcudart.so.12")
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    s, g = ctypes.c_void_p(), ctypes.c_void_p()
    assert rt.cudaStreamCreateWithFlags(ctypes.byref(s), 1) == 0
    assert rt.cudaStreamBeginCapture(s, 2) == 0                  # relaxed: other calls of the process go on
    st = tq.call_status("tq_cache_status", word.data_ptr(), s)
    left = rt.cudaPeekAtLastError()
    rt.cudaStreamEndCapture(s, ctypes.byref(g))
    rt.cudaGetLastError()
    if g.value:
        rt.cudaGraphDestroy(g)
    assert rt.cudaStreamDestroy(s) == 0
    assert st == tq.TQ_ERR_CUDA and left == 0


def test_reports_of_another_device(tq):
    """check() waits for a stream of the current device, so the status word has to be there (here it is on the host)."""
    for cls in (tq.PageTable, tq.KV4Cache):
        x = object.__new__(cls)
        x._status = torch.ones(1, dtype=torch.int32)
        with pytest.raises(ValueError, match="cpu"):
            x.check()
        assert int(x._status) == 1
