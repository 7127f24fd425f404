"""GPU parity of the paged 4-bit cache at the ends of what it may hold."""

import numpy as np
import pytest

from oracle import kv4 as o
from tests.test_gpu_kv4 import attention_tolerance, dev

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]


@pytest.fixture(scope="module")
def tq():
    from kv_cache_vector_15_b200 import tq as _tq
    return _tq


def filled(tq, rng, lens, k, v, ps):
    """A cache that holds the rows k, v (one sequence after the other) on pages
    in random order, and its table."""
    H, d = k.shape[1:]
    need = [-(-n // ps) for n in lens]
    perm = rng.permutation(sum(need) + 1).astype(np.int32)
    table = np.zeros((len(lens), max(need)), np.int32)
    at, slots = 0, []
    for i, n in enumerate(lens):
        table[i, :need[i]] = perm[at:at + need[i]]
        at += need[i]
        slots.append(table[i, np.arange(n) // ps].astype(np.int64) * ps + np.arange(n) % ps)
    C = tq.KV4Cache.empty(sum(need) + 1, H, d, ps)
    C.append(dev(k), dev(v), dev(np.concatenate(slots)))
    C.check()
    return C, dev(table)


def spoil(C, table, seq, part, tokens, head, group):
    """NaN pairs for a group of a head's rows, written by hand (part 0: K, 1: V)."""
    nb, d = C.page_size // 16, C.d
    for t in tokens:
        page, at = int(table[seq, t // C.page_size]), t % C.page_size
        pair = (head * nb + at // 16) * 18 * d + part * 9 * d + 8 * d + at % 16 * (d // 16) + 4 * group
        C.pool[page, pair:pair + 4] = torch.tensor([0xff, 0x7f] * 2, dtype=torch.uint8, device="cuda")


def small_values(C, dtype, many, n):
    """What that bound leaves out, for outputs that are small beside the values
    of their group: the few-row kernel's codes enter as 16 + c and c - 31 (bf16
    rows), so the 2^-17 that p s is off by counts for up to 31 s and not for
    |c - 8| s; the many-row kernel's p, binary16 with 2^7 for the largest, is
    off by 2^-25 where it is below 2^-14, 2^-32 of the largest for each key."""
    H, d, ps = C.kv_heads, C.d, C.page_size
    s, z = (np.stack([o.read_rows(C.pool.cpu().numpy(), np.arange(C.pool.shape[0]), C.pool.shape[0] * ps, 1, h, H, d, ps)[i]
                      for h in range(H)]).astype(np.float64) for i in (1, 2))
    if many:
        return n * 2.0 ** -32 * np.nanmax(np.abs(z) + 15 * s)
    return 31 * 2.0 ** -17 * np.nanmax(s) if dtype == "bf16" else 0.0


def compare(tq, C, table, lens, nq, q, causal=True, window=0, max_q=None):
    """The call against the oracle: NaN where the oracle has NaN, the rest within the derived bounds."""
    cu = np.concatenate([[0], np.cumsum(nq)]).astype(np.int32)
    hint = max_q or max(nq)
    out, lse = C.attention(q, table, dev(np.array(lens, np.int32)), dev(cu), hint, causal=causal, window=window, return_lse=True)
    C.check()
    dtype, d = "bf16" if q.dtype == torch.bfloat16 else "f32", q.shape[2]
    many = dtype == "bf16" and hint * q.shape[1] // C.kv_heads > 16
    with np.errstate(invalid="ignore", over="ignore"):
        ref = o.attention(q.double().cpu().numpy(), C.pool.cpu().numpy(), table.cpu().numpy(), lens, cu, C.kv_heads, C.page_size,
                          d ** -0.5, causal, window)
        tol, ltol = attention_tolerance(ref, max(lens), dtype, many, d)
        tol = tol + small_values(C, dtype, many, max(lens))
    got, gl = out.double().cpu().numpy(), lse.double().cpu().numpy()
    nan, lnan = np.isnan(ref[0]), np.isnan(ref[1])
    assert np.array_equal(np.isnan(got), nan), (np.isnan(got).sum(), nan.sum())
    assert np.array_equal(np.isnan(gl), lnan)
    inf = np.isneginf(ref[1])
    assert np.array_equal(np.isneginf(gl), inf)
    off = np.abs(got - ref[0])[~nan] / tol[~nan]
    assert off.size == 0 or off.max() <= 1, off.max()
    loff = (np.abs(gl - ref[1]) / ltol)[~(lnan | inf)]
    assert loff.size == 0 or loff.max() <= 1, loff.max()
    return nan, lnan


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("nq,dtype", [(1, "bf16"), (3, "f32"), (40, "bf16")])
def test_groups_that_span_the_whole_range(tq, d, nq, dtype):
    """Groups from -65504 to 65504 (scales of 8736, codes times scale past
    binary16's end): every kernel reads the values that the codes stand for.
    Spans on both sides of 8 s = 65504 and of z + 15 s = 65504."""
    rng = np.random.default_rng(d + nq)
    n, H = 90, 2
    x = np.linspace(-65504, 65504, 64)[None, None, None].repeat(2 * n * H * (d // 64), 0).reshape(2, n, H, d // 64, 64)
    x = rng.permuted(x, axis=-1) * np.where(rng.random((2, n, H, d // 64, 1)) < 0.5, 1.0, rng.uniform(0.9, 1, (2, n, H, d // 64, 1)))
    k, v = x.reshape(2, n, H, d).astype(np.float32)
    C, table = filled(tq, rng, [n], k, v, 16)
    q = dev((rng.standard_normal((nq, 2 * H, d)) * 2e-5 * (128 / d) ** 0.5).astype(np.float32)).to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    for causal in (True, False):
        nan, _ = compare(tq, C, table, [n], [nq], q, causal)
        assert not nan.any()


def cache_with_nan(tq, rng, d, dtype, lens, nq, where):
    """Two kv heads of random rows, NaN pairs in head 0 of the first sequence:
    a key three quarters through the new tokens, values before, among and behind them."""
    H, g, n0 = 2, 2, lens[0]
    k, v = rng.standard_normal((2, sum(lens), H, d)).astype(np.float32)
    C, table = filled(tq, rng, lens, k, v, 32)
    if where != "v":
        spoil(C, table, 0, 0, [n0 - nq[0] + nq[0] * 3 // 4], 0, d // 64 - 1)
    if where != "k":
        for t in (n0 - 1, n0 - nq[0] + nq[0] // 2, n0 - nq[0] - 10, 3):
            spoil(C, table, 0, 1, [t], 0, int(rng.integers(0, d // 64)))
    q = dev((1.5 * rng.standard_normal((sum(nq), H * g, d))).astype(np.float32)).to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    return C, table, q


@pytest.mark.parametrize("d,dtype,lens,nq,window", [
    (128, "bf16", [40, 130], [1, 1], 0), (128, "bf16", [130, 40], [4, 3], 0), (64, "f32", [130, 40], [4, 3], 0),
    (256, "f32", [130, 40], [7, 3], 5), (128, "bf16", [300, 77], [60, 40], 0), (128, "bf16", [300, 77], [60, 40], 40),
    (64, "bf16", [300, 77], [60, 40], 40), (256, "bf16", [300, 77], [60, 40], 40), (128, "bf16", [3000, 77], [200, 1], 700),
    (256, "bf16", [3000, 77], [200, 1], 0)])
@pytest.mark.parametrize("where", ["k", "v", "both"])
def test_nan_in_the_cache_reaches_the_rows_that_see_it(tq, d, dtype, lens, nq, window, where):
    """And no others: a key's NaN all of a row's outputs, a value's NaN the
    coordinates of its group; rows whose mask leaves the token out, other heads
    and other sequences do not change."""
    C, table, q = cache_with_nan(tq, np.random.default_rng(sum(lens) + d + window), d, dtype, lens, nq, where)
    nan, _ = compare(tq, C, table, lens, nq, q, True, window)
    assert nan.any() and not nan.all()
    nan, _ = compare(tq, C, table, lens, nq, q, False)
    assert nan.any() and not nan.all()


def test_nan_behind_a_weight_that_is_zero_in_fp32(tq):
    """A NaN value counts however small its token's weight is, inside a run of keys and at its edge."""
    rng = np.random.default_rng(8)
    for n, nq, dtype in ((41, 1, "bf16"), (64, 1, "bf16"), (77, 4, "f32"), (300, 20, "bf16")):
        k, v = rng.standard_normal((2, n, 1, 64)).astype(np.float32)
        k[:, :, 0] = 8.0
        for t in (2, n - 1):
            low = k.copy()
            low[t, 0, 0] = -8.0
            C, table = filled(tq, rng, [n], low, v, 16)
            spoil(C, table, 0, 1, [t], 0, 0)
            q = torch.zeros((nq, 2, 64), device="cuda", dtype=torch.bfloat16 if dtype == "bf16" else torch.float32)
            q[:, :, 0] = 300.0
            nan, lnan = compare(tq, C, table, [n], [nq], q, causal=False)
            assert nan.all() and not lnan.any()


@pytest.mark.parametrize("nq,dtype", [(1, "bf16"), (3, "f32"), (40, "bf16")])
@pytest.mark.parametrize("what", [np.nan, np.inf, -np.inf])
def test_rows_of_queries_that_are_not_finite(tq, nq, dtype, what):
    """A query with a NaN or an infinity gives NaN (its logits are infinite or
    NaN), also where all of its logits are -infinity; the rows beside it stay as they are."""
    rng = np.random.default_rng(nq)
    lens, H, g, d = [77, 90], 2, 3, 64
    k, v = (rng.standard_normal((2, sum(lens), H, d)) + 9.0).astype(np.float32)      # every key is positive
    C, table = filled(tq, rng, lens, k, v, 16)
    q = rng.standard_normal((2 * nq, H * g, d)).astype(np.float32)
    q[nq - 1, 1, 7], q[nq, 4, 0] = what, what
    nan, lnan = compare(tq, C, table, lens, [nq, nq], dev(q).to(torch.bfloat16 if dtype == "bf16" else torch.float32), False)
    assert nan.all(-1).sum() == 2 and lnan.sum() == 2


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_nan_rows_stay_nan(tq, dtype):
    """A NaN coordinate makes its group of 64 NaN: codes 0 with a pair of NaN;
    other groups, rows and heads are what they were without it."""
    rng = np.random.default_rng(3)
    n, H, d, ps = 40, 3, 128, 16
    x = rng.standard_normal((n, H, d)).astype(np.float32)
    clean = x.copy()
    x[4, 1, 70] = np.nan
    x[5, 2, :64] = np.nan
    x[6, 0, 3], x[6, 0, 4] = np.nan, np.inf
    x[7, 0, [64, 127]] = [-np.inf, np.nan]
    x[8, 1, ::64] = -np.nan
    bad = np.isnan(x).reshape(n, H, 2, 64).any(-1)
    tt = torch.bfloat16 if dtype == "bf16" else torch.float32
    C = tq.KV4Cache.empty(4, H, d, ps)
    slots = dev(rng.permutation(4 * ps)[:n].astype(np.int64))
    kv, vv = C.append(dev(x).to(tt), dev(clean).to(tt), slots, return_values=True)
    _, plain = C.append(dev(clean).to(tt), dev(x).to(tt), slots, return_values=True)      # over the rows before
    C.check()
    spread = np.repeat(bad, 64, -1)
    assert np.array_equal(torch.isnan(kv).cpu().numpy(), spread) and np.array_equal(torch.isnan(plain).cpu().numpy(), spread)
    assert torch.equal(kv[dev(~spread)], vv[dev(~spread)]) and not torch.isnan(vv).any()
    kk, vb = C.dequant(slots, out_dtype=tt)
    assert torch.equal(kk, vv) and np.array_equal(torch.isnan(vb).cpu().numpy(), spread)
    want = np.zeros(tuple(C.pool.shape), np.uint8)
    for part, y in ((0, clean), (1, x)):
        c, s, z = o.quantize(dev(y).to(tt).float().cpu().numpy())
        for t in range(n):
            for h in range(H):
                o.write_slot(want, int(slots[t]), part, h, c[t, h], s[t, h], z[t, h], H, d, ps)
    assert np.array_equal(C.pool.cpu().numpy(), want)


def test_quotients_that_64_bits_do_not_tell_from_a_border(tq):
    """x a little beside zero, zero a border between two codes: x - z is the
    border itself in 64 bits, the exact quotient is not."""
    C = tq.KV4Cache.empty(15, 1, 64, 16)
    tiny = np.float32([2.0 ** -60, 2.0 ** -149, 1e-30, 0.0, -0.0, -1e-30, -2.0 ** -149, -2.0 ** -60])
    x = np.empty((15, 1, 64), np.float32)
    want = np.empty((15, 64))
    for k in range(15):
        z = -(2.0 * k + 1)                                       # s = 2: zero is the border behind code k
        x[k, 0] = np.concatenate([[z, z + 30], np.resize(tiny, 62)])
        up = x[k, 0] > 0
        want[k] = z + 2 * np.where(up, k + 1, k)
        want[k][x[k, 0] == 0] = z + 2 * (k + k % 2)              # a tie: the even code
        want[k, :2] = z, z + 30
    got, _ = C.append(dev(x), dev(x), torch.arange(15, device="cuda"), return_values=True)
    assert np.array_equal(got.double().cpu().numpy()[:, 0], want)
    c, s, z = o.quantize(x)
    assert np.array_equal(o.values(c, s, z)[:, 0], want)


@pytest.mark.parametrize("nq,dtype,n", [(1, "bf16", 5000), (3, "f32", 700), (5, "bf16", 90), (60, "bf16", 3000)])
def test_outputs_in_the_place_of_the_queries(tq, nq, dtype, n):
    """out may be q: a row's output is written behind all reads of its query,
    by one worker, or by the join behind all workers."""
    rng = np.random.default_rng(n)
    lens, H, g, d = [n, 40, n // 3], 2, 4, 128
    k, v = rng.standard_normal((2, sum(lens), H, d)).astype(np.float32)
    C, table = filled(tq, rng, lens, k, v, 16)
    q = dev(rng.standard_normal((3 * nq, H * g, d)).astype(np.float32)).to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    cu = torch.arange(4, device="cuda", dtype=torch.int32) * nq
    args = (table, dev(np.array(lens, np.int32)), cu, nq)
    want = C.attention(q, *args)
    for _ in range(5):
        x = q.clone()
        assert C.attention(x, *args, out=x) is not None and torch.equal(x, want)
    C.check()
