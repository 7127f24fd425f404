"""The paged 4-bit cache, the query / key step before it and the page table, in
fp64 NumPy (parity status: pinned by ``tests/test_oracle_kv4.py``).

Written from the definitions in ``include/tq.h``; shares no code with the library.
"""

from __future__ import annotations

import math

import numpy as np

GROUP = 64
BLOCK = 16


# ------------------------------------------------------------- the format --

def quantize(x):
    """Rows [..., d] to (codes int [..., d], scale f16 [..., d / 64], zero f16
    [..., d / 64]); a group with a NaN: codes 0, scale and zero the NaN 0x7fff."""
    x = np.clip(np.asarray(x, np.float32), -65504, 65504)
    g = x.reshape(*x.shape[:-1], x.shape[-1] // GROUP, GROUP)
    zero = (g.min(-1) + np.float32(0)).astype(np.float16)
    span = (g.max(-1) - zero.astype(np.float32)).astype(np.float32)
    scale = (np.where(span > 0, span, np.float32(0)) / np.float32(15)).astype(np.float32).astype(np.float16)
    for pair in (scale, zero):
        pair.view(np.uint16)[np.isnan(g).any(-1)] = 0x7fff
    s, z = scale.astype(np.float64)[..., None], zero.astype(np.float64)[..., None]
    # the exact quotient, to the nearest: a code per border z + (k + 1/2) s (exact in fp64) that x lies behind; on the
    # border itself the even one of the two codes
    x64, codes = g.astype(np.float64), np.zeros(g.shape, np.int64)
    for k in range(15):
        border = z + (k + 0.5) * s
        codes += (s > 0) & ((x64 > border) | ((x64 == border) & (k % 2 == 1)))
    return codes.reshape(x.shape), scale, zero


def values(codes, scale, zero):
    """What codes stand for, fp64 [..., d]."""
    g = codes.reshape(*codes.shape[:-1], codes.shape[-1] // GROUP, GROUP).astype(np.float64)
    v = zero.astype(np.float64)[..., None] + scale.astype(np.float64)[..., None] * g
    return v.reshape(codes.shape)


def page_bytes(d, kv_heads, page_size):
    return kv_heads * (page_size // BLOCK) * 18 * d


def write_slot(pool, slot, part, head, codes, scale, zero, kv_heads, d, page_size):
    """One row (part 0: K, 1: V) into pool (uint8 [n_pages, page_bytes]), byte by byte."""
    page, at = divmod(int(slot), page_size)
    base = (head * (page_size // BLOCK) + at // BLOCK) * 18 * d + part * 9 * d
    t = at % BLOCK
    row = pool[page]
    for i in range(d // 2):
        row[base + t * (d // 2) + i] = int(codes[2 * i]) | (int(codes[2 * i + 1]) << 4)
    pair = np.stack([scale, zero], -1).astype(np.float16).reshape(-1).view(np.uint8)
    row[base + 8 * d + t * (d // 16): base + 8 * d + (t + 1) * (d // 16)] = pair


def read_rows(pool, pages, n, part, head, kv_heads, d, page_size):
    """(codes [n, d], scale [n, d / 64], zero) of the first n tokens of a sequence's pages."""
    nb = page_size // BLOCK
    p = pool.reshape(pool.shape[0], kv_heads, nb, 18 * d)[np.asarray(pages, np.int64), head]     # [P, nb, 18 d]
    p = p.reshape(-1, 18 * d)[:, part * 9 * d:(part + 1) * 9 * d]
    raw = p[:, :8 * d].reshape(-1, d // 2)[:n]
    codes = np.empty((raw.shape[0], d), np.int64)
    codes[:, 0::2], codes[:, 1::2] = raw & 15, raw >> 4
    pair = np.ascontiguousarray(p[:, 8 * d:]).view(np.float16).reshape(-1, d // GROUP, 2)[:n]
    return codes, pair[..., 0], pair[..., 1]


# -------------------------------------------------------------- attention --

def attention(q, pool, table, lens, cu_q, kv_heads, page_size, scale, causal=True, window=0):
    """q fp64 [T, q_heads, d] against the pool; returns out fp64 [T, q_heads, d]
    and lse [T, q_heads] (tokens of no sequence: NaN), and per output the
    bounds that tolerances are made of: ``mag`` [T, q_heads, d] = sum_t p_t
    (s |c - 8| + |z + 8 s|), ``err`` [T, q_heads] = the largest over seen
    tokens of scale * sum_d |q_d| (s |c| + |z|), and ``qerr`` likewise of
    scale * max_d |q_d| * sum_d s c."""
    T, hq, d = q.shape
    g = hq // kv_heads
    out = np.full(q.shape, np.nan)
    lse = np.full((T, hq), np.nan)
    mag, err, qerr = np.zeros(q.shape), np.zeros((T, hq)), np.zeros((T, hq))
    for i, n in enumerate(lens):
        q0, q1 = int(cu_q[i]), int(cu_q[i + 1])
        nq, n = q1 - q0, int(n)
        if nq == 0:
            continue
        for h in range(kv_heads):
            pages = table[i][:-(-n // page_size)]
            ck, sk, zk = read_rows(pool, pages, n, 0, h, kv_heads, d, page_size)
            cv, sv, zv = read_rows(pool, pages, n, 1, h, kv_heads, d, page_size)
            K, V = values(ck, sk, zk), values(cv, sv, zv)
            up = lambda a: np.repeat(a.astype(np.float64), GROUP, -1)  # noqa: E731
            absk = up(sk) * ck + np.abs(up(zk))
            absv = up(sv) * np.abs(cv - 8) + np.abs(up(zv) + 8 * up(sv))
            for j in range(nq):
                pos = n - nq + j
                hi = pos if causal else n - 1
                lo = max(0, pos - window + 1) if window else 0
                for e in range(g):
                    t, r = q0 + j, h * g + e
                    if hi < lo or n == 0:
                        out[t, r], lse[t, r] = 0.0, -np.inf
                        continue
                    x = K[lo:hi + 1] @ q[t, r] * scale
                    m = x.max()
                    w = np.exp(x - m)
                    lse[t, r] = m + math.log(w.sum())
                    w /= w.sum()
                    out[t, r] = w @ V[lo:hi + 1]
                    mag[t, r] = w @ absv[lo:hi + 1]
                    err[t, r] = abs(scale) * (absk[lo:hi + 1] @ np.abs(q[t, r])).max()
                    qerr[t, r] = abs(scale) * np.abs(q[t, r]).max() * (up(sk) * ck)[lo:hi + 1].sum(-1).max()
    return out, lse, mag, err, qerr


# ----------------------------------------------------- norm and rotation --

def norm_rope(x, weight, eps, positions, inv_freq, interleaved, axis):
    """x fp64 [n, heads, d]; positions int [axes, n]; returns fp64 rows and the
    size |y_a| + |y_b| that the rotation's rounding errors scale with."""
    n, _, d = x.shape
    y = x / np.sqrt(np.mean(x * x, -1, keepdims=True) + eps) * (1.0 if weight is None else weight)
    out, size = y.copy(), np.abs(y)
    half = len(inv_freq)
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        t = positions[axis[i]].astype(np.float64) * inv_freq[i]
        c, s = np.cos(t)[:, None], np.sin(t)[:, None]
        out[..., a] = y[..., a] * c - y[..., b] * s
        out[..., b] = y[..., a] * s + y[..., b] * c
        size[..., a] = size[..., b] = np.abs(y[..., a]) + np.abs(y[..., b])
    return out, size


# ------------------------------------------------------------------ pages --

class Pages:
    """The page table as plain lists of Python's arithmetic."""

    def __init__(self, table, lens, refs, page_size):
        self.table, self.lens, self.refs = np.array(table), np.array(lens), np.array(refs)
        self.page_size = page_size

    def copy(self):
        return Pages(self.table, self.lens, self.refs, self.page_size)

    def _pages(self, n):
        return -(-int(n) // self.page_size)

    def extend(self, seqs, more):
        """The new tokens' slots; None (and nothing done) where the call cannot be done."""
        if len(set(seqs)) < len(seqs) or any(not 0 <= s < len(self.lens) for s in seqs) or any(t < 0 for t in more):
            return None
        cap = self.table.shape[1] * self.page_size
        need = 0
        for s, t in zip(seqs, more):
            n = int(self.lens[s])
            if n + t > cap:
                return None
            if t and n % self.page_size and self.refs[self.table[s, self._pages(n) - 1]] != 1:
                return None
            need += self._pages(n + t) - self._pages(n)
        free = [p for p in range(len(self.refs)) if self.refs[p] <= 0]
        if need > len(free):
            return None
        slots = []
        for s, t in zip(seqs, more):
            n = int(self.lens[s])
            for p in range(self._pages(n), self._pages(n + t)):
                self.table[s, p] = free.pop(0)
                self.refs[self.table[s, p]] = 1
            slots += [int(self.table[s, k // self.page_size]) * self.page_size + k % self.page_size for k in range(n, n + t)]
            self.lens[s] = n + t
        return slots

    def fork(self, src, dst):
        ok = all(0 <= x < len(self.lens) for x in list(src) + list(dst)) and len(set(dst)) == len(dst)
        if not ok or any(self.lens[x] for x in dst):
            return None
        part = [int(self.lens[x]) % self.page_size != 0 for x in src]
        free = [p for p in range(len(self.refs)) if self.refs[p] <= 0]
        if sum(part) > len(free):
            return None
        lens, moves = [int(self.lens[x]) for x in src], []
        for a, b, n, p in zip(src, dst, lens, part):
            full = n // self.page_size
            self.table[b] = -1
            for k in range(full):
                self.table[b, k] = self.table[a, k]
                self.refs[self.table[a, k]] += 1
            if p:
                self.table[b, full] = free.pop(0)
                self.refs[self.table[b, full]] = 1
                moves.append((int(self.table[a, full]), int(self.table[b, full])))
            self.lens[b] = n
        return moves

    def free(self, seqs):
        if any(not 0 <= s < len(self.lens) for s in seqs):
            return False
        for s in set(seqs):
            for k in range(self._pages(self.lens[s])):
                self.refs[self.table[s, k]] -= 1
            self.table[s], self.lens[s] = -1, 0
        return True

    def compact(self):
        used = [p for p in range(len(self.refs)) if self.refs[p] > 0]
        holes = [p for p in range(len(used)) if self.refs[p] <= 0]
        high = [p for p in used if p >= len(used)]
        to = dict(zip(high, holes))
        for a, b in to.items():
            self.refs[b], self.refs[a] = self.refs[a], 0
        for s in range(len(self.lens)):
            n = self._pages(self.lens[s])
            self.table[s, n:] = -1
            for k in range(n):
                self.table[s, k] = to.get(int(self.table[s, k]), int(self.table[s, k]))
        return list(zip(high, holes))
