"""Thin ctypes binding of libtq (include/tq.h).

Argument marshalling only: every step of the method runs inside libtq's CUDA
kernels.  PyTorch supplies device memory and the current CUDA stream.  If
libtq.so is missing or cannot be loaded this module raises at import time;
there is no fallback path.
"""

from __future__ import annotations

import ctypes
import math
import operator
import os
from dataclasses import dataclass

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.environ.get("TQ_LIB", os.path.join(_HERE, "libtq.so"))

if not os.path.exists(LIB_PATH):
    raise ImportError(f"libtq.so not found at {LIB_PATH}; build it with `python -m kv_cache_vector_15_b200.build`")
_lib = ctypes.CDLL(LIB_PATH)

TQ_OK, TQ_ERR_INVALID_ARG, TQ_ERR_UNSUPPORTED, TQ_ERR_NOMEM, TQ_ERR_CUDA = range(5)
TQ_BF16, TQ_F32 = 0, 1
TQ_DEQUANT_PROD, TQ_DEQUANT_MSE = 0, 1
TQ_TEST_WAIT_LIMIT, TQ_TEST_FAIL_ALLOC, TQ_TEST_FAIL_LAUNCH, TQ_TEST_FIXUP_CAP = 0, 1, 2, 3

# exported symbols, in header order
SYMBOLS = [
    "tq_host_params", "tq_init", "tq_destroy", "tq_packed_sizes", "tq_get_params", "tq_quantize_workspace_bytes",
    "tq_quantize", "tq_logits_workspace_bytes", "tq_logits", "tq_logits_noalloc", "tq_dequant", "tq_topk", "tq_logits_bf16",
    "tq_status_str", "tq_sync_status", "tq_last_error", "tq_launch_count", "tq_attention_workspace_bytes",
    "tq_attention", "tq_quantize_scatter", "tq_search_workspace_bytes", "tq_search", "tq_split_init",
    "tq_split_destroy", "tq_split_part", "tq_split_quantize_workspace_bytes", "tq_split_quantize",
    "tq_split_logits_workspace_bytes", "tq_split_logits",
    "tq_split_dequant", "tq_test_set", "tq_qk_norm_rope", "tq_kv4_page_bytes", "tq_kv4_append", "tq_kv4_dequant",
    "tq_kv4_attention_workspace_bytes", "tq_kv4_attention", "tq_pages_workspace_bytes", "tq_pages_extend",
    "tq_pages_fork", "tq_pages_free", "tq_pages_compact", "tq_pages_copy", "tq_cache_status",
]


class _Packed(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("signs", ctypes.c_void_p), ("norm", ctypes.c_void_p),
                ("rnorm", ctypes.c_void_p)]


class _KV4(ctypes.Structure):
    _fields_ = [("pool", ctypes.c_void_p), ("n_pages", ctypes.c_int64), ("d", ctypes.c_int32),
                ("kv_heads", ctypes.c_int32), ("page_size", ctypes.c_int32), ("status", ctypes.c_void_p)]


class _Pages(ctypes.Structure):
    _fields_ = [("table", ctypes.c_void_p), ("lens", ctypes.c_void_p), ("refs", ctypes.c_void_p),
                ("n_seqs", ctypes.c_int64), ("max_pages", ctypes.c_int64), ("n_pages", ctypes.c_int64),
                ("page_size", ctypes.c_int32), ("status", ctypes.c_void_p)]


_vp, _i32, _i64, _u64, _sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_uint64, ctypes.c_size_t
_sig = {
    "tq_host_params": (_i32, [_i32, _i32, _i32, _u64, _vp, _vp, _vp, _vp]),
    "tq_init": (_i32, [_i32, _i32, _i32, _u64, ctypes.POINTER(_vp)]),
    "tq_destroy": (_i32, [_vp]),
    "tq_packed_sizes": (_i32, [_vp, _i64, ctypes.POINTER(_sz), ctypes.POINTER(_sz)]),
    "tq_get_params": (_i32, [_vp, _vp, _vp, _vp, _vp]),
    "tq_quantize_workspace_bytes": (_sz, [_vp, _i64]),
    "tq_quantize": (_i32, [_vp, _vp, _i32, _i64, _i64, _Packed, _vp, _sz, _vp]),
    "tq_quantize_scatter": (_i32, [_vp, _vp, _i32, _i64, _i64, _vp, _i64, _Packed, _vp]),
    "tq_logits_workspace_bytes": (_sz, [_vp, _i64, _i32, _i64]),
    "tq_logits": (_i32, [_vp, _vp, _i32, _i64, _i32, _Packed, _i64, _vp, _vp, _sz, _vp]),
    "tq_logits_noalloc": (_i32, [_vp, _vp, _i32, _i64, _i32, _Packed, _i64, _vp, _vp]),
    "tq_dequant": (_i32, [_vp, _Packed, _i64, _vp, _i32, _i32, _vp]),
    "tq_attention_workspace_bytes": (_sz, [_vp, _i64, _i32, _i64]),
    "tq_attention": (_i32, [_vp, _vp, _i32, _i64, _i32, _Packed, _Packed, _i64, ctypes.c_float, _i32, _vp, _vp, _sz,
                            _vp]),
    "tq_search_workspace_bytes": (_sz, [_vp, _i64, _i64, _i32]),
    "tq_search": (_i32, [_vp, _vp, _i32, _i64, _Packed, _i64, _i32, _vp, _vp, _vp, _sz, _vp]),
    "tq_split_init": (_i32, [_i32, _i32, _i32, _i32, _u64, ctypes.POINTER(_vp)]),
    "tq_split_destroy": (_i32, [_vp]),
    "tq_split_part": (_i32, [_vp, _i32, ctypes.POINTER(_vp)]),
    "tq_split_quantize_workspace_bytes": (_sz, [_vp, _i64]),
    "tq_split_quantize": (_i32, [_vp, _vp, _i32, _i64, _i64, _Packed, _Packed, _vp, _sz, _vp]),
    "tq_split_logits_workspace_bytes": (_sz, [_vp, _i64, _i32, _i64]),
    "tq_split_logits": (_i32, [_vp, _vp, _i32, _i64, _i32, _Packed, _Packed, _i64, _vp, _vp, _sz, _vp]),
    "tq_split_dequant": (_i32, [_vp, _Packed, _Packed, _i64, _vp, _i32, _i32, _vp]),
    "tq_topk": (_i32, [_vp, _i64, _i64, _i32, _vp, _vp, _vp]),
    "tq_logits_bf16": (_i32, [_vp, _vp, _i64, _i32, _i64, _i32, _vp, _vp]),
    "tq_status_str": (ctypes.c_char_p, [_i32]),
    "tq_sync_status": (_i32, [_vp, _vp]),
    "tq_last_error": (ctypes.c_char_p, []),
    "tq_launch_count": (_u64, []),
    "tq_test_set": (_i32, [_i32, _i64]),
    "tq_qk_norm_rope": (_i32, [_vp, _i64, _i32, _vp, _i64, _i32, _i32, _i64, _i32, _vp, _vp, ctypes.c_float, _vp, _i32,
                               _i32, _i32, _vp, _vp, _vp, _i64, _vp, _i64, _vp]),
    "tq_kv4_page_bytes": (_sz, [_i32, _i32, _i32]),
    "tq_kv4_append": (_i32, [_KV4, _vp, _i64, _vp, _i64, _i32, _i64, _vp, _vp, _vp, _vp]),
    "tq_kv4_dequant": (_i32, [_KV4, _vp, _i64, _vp, _vp, _i32, _vp]),
    "tq_kv4_attention_workspace_bytes": (_sz, [_KV4, _i32, _i32, _i64, _i64, _i32]),
    "tq_kv4_attention": (_i32, [_KV4, _vp, _i32, _i64, _i32, _i64, _i64, _vp, _i32, _vp, _i64, _vp, ctypes.c_float,
                                _i32, _i32, _vp, _vp, _vp, _sz, _vp]),
    "tq_pages_workspace_bytes": (_sz, [_Pages, _i64]),
    "tq_pages_extend": (_i32, [_Pages, _Pages, _i64, _vp, _vp, _vp, _i64, _vp, _sz, _vp]),
    "tq_pages_fork": (_i32, [_Pages, _Pages, _i64, _vp, _vp, _vp, _vp, _sz, _vp]),
    "tq_pages_free": (_i32, [_Pages, _Pages, _i64, _vp, _vp, _sz, _vp]),
    "tq_pages_compact": (_i32, [_Pages, _Pages, _vp, _vp, _sz, _vp]),
    "tq_pages_copy": (_i32, [_vp, _i64, _i64, _i64, _i64, _vp, _i64, _vp]),
    "tq_cache_status": (_i32, [_vp, _vp]),
}
for _name, (_res, _args) in _sig.items():
    _f = getattr(_lib, _name)
    _f.restype = _res
    _f.argtypes = _args


class TQError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        msg = _lib.tq_last_error().decode(errors="replace")
        super().__init__(f"{where}: {_lib.tq_status_str(status).decode()} ({msg})")


def _check(status: int, where: str):
    if status != TQ_OK:
        raise TQError(status, where)


def test_set(knob: int, value: int):
    """Process-wide test setting (tq_test_set): wait limit of the d = 128
    quantize kernel, or injected host-side allocation / launch failures."""
    _check(_lib.tq_test_set(knob, value), "tq_test_set")


def launch_count() -> int:
    """Kernel launches libtq has issued in this process."""
    return int(_lib.tq_launch_count())


def host_params(d: int, b: int, m: int, seed: int = 0):
    """Parameters derived on the host (no CUDA): centroids, thresholds (fp32),
    D (int8), S (binary16 as numpy float16, [m, d']), where d' is d padded to
    the next power of two."""
    L = 1 << (b - 1)
    dp = 1 << (d - 1).bit_length() if d > 0 else 0
    c = np.zeros(L, np.float32)
    t = np.zeros(L - 1, np.float32)
    D = np.zeros(max(dp, 1), np.int8)
    S = np.zeros(max(m * dp, 1), np.uint16)
    _check(_lib.tq_host_params(d, b, m, seed & (2**64 - 1), c.ctypes.data, t.ctypes.data, D.ctypes.data,
                               S.ctypes.data), "tq_host_params")
    return c, t, D, S.view(np.float16).reshape(m, dp)


def _ptr(t) -> int:
    return 0 if t is None else int(t.data_ptr())


def _stream(stream) -> int:
    if stream is not None:
        return int(stream.cuda_stream)
    import torch
    # torch.cuda.current_stream().cuda_stream without the Stream object, whose making takes 3 us
    return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())


def _dtype_code(t) -> int:
    import torch
    if t.dtype == torch.bfloat16:
        return TQ_BF16
    if t.dtype == torch.float32:
        return TQ_F32
    raise TypeError(f"unsupported dtype {t.dtype}")


@dataclass
class Packed:
    """Packed rows: codes [N, d(b-1)/8] u8, signs [N, m/8] u8, norm [N], rnorm [N] f32."""

    codes: "object"
    signs: "object"
    norm: "object"
    rnorm: "object"

    @property
    def n_rows(self) -> int:
        return int(self.norm.shape[0])

    def c(self) -> _Packed:
        return _Packed(_ptr(self.codes), _ptr(self.signs), _ptr(self.norm), _ptr(self.rnorm))

    def nbytes(self) -> int:
        return sum(int(t.numel() * t.element_size()) for t in (self.codes, self.signs, self.norm, self.rnorm))

    def rows(self, start: int, stop: int) -> "Packed":
        """Rows [start, stop) as views of the same storage."""
        return Packed(self.codes[start:stop], self.signs[start:stop], self.norm[start:stop], self.rnorm[start:stop])

    def to_numpy(self) -> dict:
        return {k: getattr(self, k).cpu().numpy() for k in ("codes", "signs", "norm", "rnorm")}

    @staticmethod
    def from_numpy(p: dict, device="cuda") -> "Packed":
        import torch
        return Packed(*(torch.from_numpy(np.ascontiguousarray(p[k])).to(device)
                        for k in ("codes", "signs", "norm", "rnorm")))


class TurboQuant:
    """One parameter set (d, b, m, seed) on the current CUDA device."""

    def __init__(self, d: int, b: int, m: int, seed: int = 0):
        self.d, self.b, self.m, self.seed = d, b, m, seed
        # rows of a length that is not a power of two are zero-padded to the next one
        self.d_pad = 1 << (d - 1).bit_length()
        h = _vp()
        _check(_lib.tq_init(d, b, m, seed & (2**64 - 1), ctypes.byref(h)), "tq_init")
        self._h = h
        cb, sb = _sz(), _sz()
        _check(_lib.tq_packed_sizes(h, 1, ctypes.byref(cb), ctypes.byref(sb)), "tq_packed_sizes")
        self.codes_bytes, self.signs_bytes = cb.value, sb.value

    def close(self):
        if getattr(self, "_h", None):
            _lib.tq_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    @property
    def handle(self):
        return self._h

    @property
    def row_bytes(self) -> int:
        return self.codes_bytes + self.signs_bytes + 8

    def params(self):
        L = 1 << (self.b - 1)
        c = np.zeros(L, np.float32)
        t = np.zeros(L - 1, np.float32)
        D = np.zeros(self.d_pad, np.int8)
        S = np.zeros(self.m * self.d_pad, np.uint16)
        _check(_lib.tq_get_params(self._h, c.ctypes.data, t.ctypes.data, D.ctypes.data, S.ctypes.data),
               "tq_get_params")
        return c, t, D, S.view(np.float16).reshape(self.m, self.d_pad)

    def empty_packed(self, n_rows: int, device="cuda") -> Packed:
        import torch
        return Packed(torch.empty((n_rows, self.codes_bytes), dtype=torch.uint8, device=device),
                      torch.empty((n_rows, self.signs_bytes), dtype=torch.uint8, device=device),
                      torch.empty((n_rows,), dtype=torch.float32, device=device),
                      torch.empty((n_rows,), dtype=torch.float32, device=device))

    def quantize_workspace_bytes(self, n_rows: int) -> int:
        return int(_lib.tq_quantize_workspace_bytes(self._h, n_rows))

    def quantize(self, x, out: Packed | None = None, workspace=None, stream=None) -> Packed:
        """x: [N, d] (or [N, ld] with ld >= d) bf16/fp32 CUDA tensor, unit stride in the last dim."""
        import torch
        assert x.dim() == 2 and x.stride(1) == 1
        n = x.shape[0]
        if out is None:
            out = self.empty_packed(n, x.device)
        need = self.quantize_workspace_bytes(n)
        if need and workspace is None:
            workspace = torch.empty(need, dtype=torch.uint8, device=x.device)
        wbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
        _check(_lib.tq_quantize(self._h, _ptr(x), _dtype_code(x), n, x.stride(0), out.c(), _ptr(workspace), wbytes,
                                _stream(stream)), "tq_quantize")
        return out

    def sync_status(self, stream=None):
        """Wait for the stream and raise if a kernel's bounded wait ran out."""
        _check(_lib.tq_sync_status(self._h, _stream(stream)), "tq_sync_status")

    def workspace_bytes(self, n_sets: int, g: int, n_keys: int) -> int:
        return int(_lib.tq_logits_workspace_bytes(self._h, n_sets, g, n_keys))

    def logits(self, q, keys: Packed, n_sets: int, g: int, n_keys: int, out=None, workspace=None,
               stream=None):
        """q: [n_sets*g, d] bf16/fp32; keys: n_sets*n_keys packed rows; returns [n_sets, g, n_keys] fp32."""
        import torch
        if out is None:
            out = torch.empty((n_sets, g, n_keys), dtype=torch.float32, device=q.device)
        need = self.workspace_bytes(n_sets, g, n_keys)
        if need and workspace is None:
            workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
        wbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
        _check(_lib.tq_logits(self._h, _ptr(q), _dtype_code(q), n_sets, g, keys.c(), n_keys, _ptr(out),
                              _ptr(workspace), wbytes, _stream(stream)), "tq_logits")
        return out

    def logits_noalloc(self, q, keys: Packed, n_sets: int, g: int, n_keys: int, out, stream=None):
        """tq_logits with the library's built-in scratch instead of a workspace;
        allocates nothing on the device (``out`` must be provided)."""
        _check(_lib.tq_logits_noalloc(self._h, _ptr(q), _dtype_code(q), n_sets, g, keys.c(), n_keys, _ptr(out),
                                      _stream(stream)), "tq_logits_noalloc")
        return out

    def dequant(self, packed: Packed, n_rows: int | None = None, out_dtype=None, mode: int = TQ_DEQUANT_PROD,
                out=None, stream=None):
        import torch
        n = packed.n_rows if n_rows is None else n_rows
        if out is None:
            out = torch.empty((n, self.d), dtype=out_dtype or torch.bfloat16, device=packed.norm.device)
        _check(_lib.tq_dequant(self._h, packed.c(), n, _ptr(out), _dtype_code(out), mode, _stream(stream)),
               "tq_dequant")
        return out


    def quantize_scatter(self, x, dest_rows, cache: Packed, stream=None) -> Packed:
        """Append: row i of x [N, d] (bf16/fp32 CUDA tensor) goes to packed row
        dest_rows[i] (int64 CUDA tensor) of ``cache``."""
        import torch
        assert x.dim() == 2 and x.stride(1) == 1
        assert dest_rows.dtype == torch.int64 and dest_rows.is_contiguous() and dest_rows.numel() == x.shape[0]
        _check(_lib.tq_quantize_scatter(self._h, _ptr(x), _dtype_code(x), x.shape[0], x.stride(0), _ptr(dest_rows),
                                        cache.n_rows, cache.c(), _stream(stream)), "tq_quantize_scatter")
        return cache

    def search_workspace_bytes(self, n_q: int, n_keys: int, k: int) -> int:
        return int(_lib.tq_search_workspace_bytes(self._h, n_q, n_keys, k))

    def search(self, q, keys: Packed, n_keys: int, k: int, idx=None, val=None, workspace=None, stream=None):
        """Vector search: per query of q [n_q, d], the k packed rows with the
        largest estimate (larger first, ties to the lower row); returns
        (idx [n_q, k] int32, val [n_q, k] fp32)."""
        import torch
        n_q = q.shape[0]
        if idx is None:
            idx = torch.empty((n_q, k), dtype=torch.int32, device=q.device)
        if val is None:
            val = torch.empty((n_q, k), dtype=torch.float32, device=q.device)
        need = self.search_workspace_bytes(n_q, n_keys, k)
        if need and workspace is None:
            workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
        wbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
        _check(_lib.tq_search(self._h, _ptr(q), _dtype_code(q), n_q, keys.c(), n_keys, k, _ptr(idx), _ptr(val),
                              _ptr(workspace), wbytes, _stream(stream)), "tq_search")
        return idx, val

    def attention_workspace_bytes(self, n_sets: int, g: int, n_keys: int) -> int:
        return int(_lib.tq_attention_workspace_bytes(self._h, n_sets, g, n_keys))

    def attention(self, q, keys: Packed, values: Packed, n_sets: int, g: int, n_keys: int, scale: float | None = None,
                  mode: int = TQ_DEQUANT_PROD, out=None, workspace=None, stream=None):
        """Decode attention from packed keys and values: [n_sets*g, d] fp32
        (softmax over each set's keys of scale * logit, times the dequantized
        values; scale defaults to 1/sqrt(d))."""
        import torch
        if scale is None:
            scale = 1.0 / math.sqrt(self.d)
        if out is None:
            out = torch.empty((n_sets * g, self.d), dtype=torch.float32, device=q.device)
        need = self.attention_workspace_bytes(n_sets, g, n_keys)
        if need and workspace is None:
            workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
        wbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
        _check(_lib.tq_attention(self._h, _ptr(q), _dtype_code(q), n_sets, g, keys.c(), values.c(), n_keys,
                                 float(scale), mode, _ptr(out), _ptr(workspace), wbytes, _stream(stream)),
               "tq_attention")
        return out


class TurboQuantSplit:
    """Fractional bit widths: channels [0, d_hi) as one instance with b_hi
    bits per coordinate, channels [d_hi, d) as another with b_lo bits (seeds
    seed and seed + 1); packed rows come in pairs (part 0, part 1)."""

    def __init__(self, d: int, d_hi: int, b_hi: int, b_lo: int, seed: int = 0):
        self.d, self.d_hi, self.b_hi, self.b_lo, self.seed = d, d_hi, b_hi, b_lo, seed
        h = _vp()
        _check(_lib.tq_split_init(d, d_hi, b_hi, b_lo, seed & (2**64 - 1), ctypes.byref(h)), "tq_split_init")
        self._h = h
        self._sizes, self._parts = [], []
        for p in (0, 1):
            ph = _vp()
            _check(_lib.tq_split_part(h, p, ctypes.byref(ph)), "tq_split_part")
            cb, sb = _sz(), _sz()
            _check(_lib.tq_packed_sizes(ph, 1, ctypes.byref(cb), ctypes.byref(sb)), "tq_packed_sizes")
            self._sizes.append((cb.value, sb.value))
            self._parts.append(ph)

    def sync_status(self, stream=None):
        """Wait for the stream and raise if a kernel of either part reported an error."""
        for ph in self._parts:
            _check(_lib.tq_sync_status(ph, _stream(stream)), "tq_sync_status")

    @property
    def row_bytes(self) -> int:
        """Packed bytes per row over both parts (codes, signs, two fp32 norms each)."""
        return sum(cb + sb + 8 for cb, sb in self._sizes)

    def logits_workspace_bytes(self, n_sets: int, g: int, n_keys: int) -> int:
        return int(_lib.tq_split_logits_workspace_bytes(self._h, n_sets, g, n_keys))

    @property
    def bits_per_coordinate(self) -> float:
        return (self.d_hi * self.b_hi + (self.d - self.d_hi) * self.b_lo) / self.d

    def close(self):
        if getattr(self, "_h", None):
            _lib.tq_split_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def empty_packed(self, n_rows: int, device="cuda"):
        import torch
        return tuple(Packed(torch.empty((n_rows, cb), dtype=torch.uint8, device=device),
                            torch.empty((n_rows, sb), dtype=torch.uint8, device=device),
                            torch.empty((n_rows,), dtype=torch.float32, device=device),
                            torch.empty((n_rows,), dtype=torch.float32, device=device)) for cb, sb in self._sizes)

    def quantize_workspace_bytes(self, n_rows: int) -> int:
        return int(_lib.tq_split_quantize_workspace_bytes(self._h, n_rows))

    def quantize(self, x, out=None, workspace=None, stream=None):
        import torch
        assert x.dim() == 2 and x.stride(1) == 1
        n = x.shape[0]
        if out is None:
            out = self.empty_packed(n, x.device)
        need = self.quantize_workspace_bytes(n)
        if need and workspace is None:
            workspace = torch.empty(need, dtype=torch.uint8, device=x.device)
        wbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
        _check(_lib.tq_split_quantize(self._h, _ptr(x), _dtype_code(x), n, x.stride(0), out[0].c(), out[1].c(),
                                      _ptr(workspace), wbytes, _stream(stream)), "tq_split_quantize")
        return out

    def logits(self, q, keys, n_sets: int, g: int, n_keys: int, out=None, workspace=None, stream=None):
        import torch
        if out is None:
            out = torch.empty((n_sets, g, n_keys), dtype=torch.float32, device=q.device)
        need = self.logits_workspace_bytes(n_sets, g, n_keys)
        if need and workspace is None:
            workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
        wbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
        _check(_lib.tq_split_logits(self._h, _ptr(q), _dtype_code(q), n_sets, g, keys[0].c(), keys[1].c(), n_keys,
                                    _ptr(out), _ptr(workspace), wbytes, _stream(stream)), "tq_split_logits")
        return out

    def dequant(self, packed, n_rows: int | None = None, out_dtype=None, mode: int = TQ_DEQUANT_PROD, out=None,
                stream=None):
        import torch
        n = packed[0].n_rows if n_rows is None else n_rows
        if out is None:
            out = torch.empty((n, self.d), dtype=out_dtype or torch.bfloat16, device=packed[0].norm.device)
        _check(_lib.tq_split_dequant(self._h, packed[0].c(), packed[1].c(), n, _ptr(out), _dtype_code(out), mode,
                                     _stream(stream)), "tq_split_dequant")
        return out


def _fixed(*names):
    """Attributes that cannot be set anew: their arrays' addresses are held beside them."""
    def add(cls):
        for name in names:
            setattr(cls, name, property(operator.attrgetter("_" + name)))
        return cls
    return add


@_fixed("inv_freq", "axis", "interleaved", "rot_dim")
class Rope:
    """A rotary position plan for qk_norm_rope: inv_freq [rot_dim / 2] (host
    numbers), pairs (i, i + rot_dim / 2) or, interleaved, (2 i, 2 i + 1); axis
    [rot_dim / 2]: which row of the positions turns pair i (None: the only one)."""

    def __init__(self, inv_freq, interleaved: bool = False, axis=None):
        self._inv_freq = np.array(inv_freq, dtype=np.float64, order="C").reshape(-1)          # its own numbers, not the caller's array
        self._axis = None if axis is None else np.array(axis, dtype=np.int32, order="C").reshape(-1)
        if self._axis is not None and self._axis.shape != self._inv_freq.shape:
            raise ValueError("axis and inv_freq differ in length")
        self._interleaved = bool(interleaved)
        self._rot_dim = 2 * self._inv_freq.size
        self._c = (self._rot_dim, int(self._interleaved), self._inv_freq.ctypes.data,
                   0 if self._axis is None else self._axis.ctypes.data)

    def __reduce__(self):                      # copies hold addresses of their own arrays
        return Rope, (self.inv_freq.copy(), self.interleaved, None if self.axis is None else self.axis.copy())


# The calls below are made once per layer and token, so their host time counts:
# their checks, outputs and workspaces are made in C++ (csrc/python/calls.cpp),
# by a module that calls the libtq loaded here.  Over ctypes a call took 11 to
# 19 us of the host, more than the kernels of a small batch take.
_calls = None


def _load_calls():
    global _calls
    import torch
    torch.cuda.init()
    from . import _calls as module                        # built with libtq: python -m kv_cache_vector_15_b200.build
    names = ("tq_qk_norm_rope", "tq_kv4_append", "tq_kv4_attention", "tq_kv4_attention_workspace_bytes",
             "tq_pages_workspace_bytes", "tq_pages_extend", "tq_pages_fork", "tq_pages_free", "tq_pages_compact",
             "tq_pages_copy")
    module.bind({n: ctypes.cast(getattr(_lib, n), _vp).value for n in names}, _check)
    _calls = module
    return module


def _on_device(*tensors):
    """Every tensor (None: not given) is on the current CUDA device."""
    import torch
    dev = torch.cuda.current_device()
    for t in tensors:
        if t is not None and t.get_device() != dev:       # -1: not on a device
            raise ValueError(f"a tensor is on {t.device}, the current device is cuda:{dev}")


def _want(x, dtype, shape, what: str):
    if x.dtype is not dtype or x.shape != shape or not x.is_contiguous():
        raise ValueError(f"{what} must be contiguous {dtype} of shape {tuple(shape)}")


def qk_norm_rope(q, k, positions, rope: Rope, q_weight=None, k_weight=None, eps: float = 1e-6, out_q=None, out_k=None,
                 stream=None):
    """RMS norm of every head of q [n, q_heads, d] and k [n, k_heads, d] (bf16
    or fp32 CUDA tensors, column ranges of a wider one are fine), times the
    weights (fp32 [d], None: ones), and the rotation by ``positions`` (int64
    [n] or [n_axes, n]); returns (out_q, out_k), new tensors unless given (q and
    k themselves: in place)."""
    return (_calls or _load_calls()).qk_norm_rope(q, k, positions, rope._c, q_weight, k_weight, eps, out_q, out_k, stream)


def kv4_page_bytes(d: int, kv_heads: int, page_size: int) -> int:
    n = int(_lib.tq_kv4_page_bytes(d, kv_heads, page_size))
    if not n:
        raise TQError(TQ_ERR_INVALID_ARG, "tq_kv4_page_bytes")
    return n


@_fixed("pool", "status", "kv_heads", "d", "page_size")
class KV4Cache:
    """One layer's keys and values in paged 4-bit form: ``pool`` is uint8
    [n_pages, kv4_page_bytes(d, kv_heads, page_size)] on the current CUDA device."""

    def __init__(self, pool, kv_heads: int, d: int, page_size: int):
        import torch
        _on_device(pool)
        _want(pool, torch.uint8, (pool.shape[0], kv4_page_bytes(d, kv_heads, page_size)), "pool")
        self._pool, self._kv_heads, self._d, self._page_size = pool, kv_heads, d, page_size
        self._status = torch.zeros(1, dtype=torch.int32, device=pool.device)
        self._c = _KV4(pool.data_ptr(), pool.shape[0], d, kv_heads, page_size, self._status.data_ptr())
        self._at = ctypes.addressof(self._c)

    @staticmethod
    def empty(n_pages: int, kv_heads: int, d: int, page_size: int, device="cuda") -> "KV4Cache":
        import torch
        return KV4Cache(torch.zeros((n_pages, kv4_page_bytes(d, kv_heads, page_size)), dtype=torch.uint8,
                                    device=device), kv_heads, d, page_size)

    def check(self, stream=None):
        """Wait for the stream and raise what kernels recorded (slots, pages or lengths out of range)."""
        _on_device(self._status)                                 # another device's stream would not be the one to wait for
        _check(_lib.tq_cache_status(_ptr(self.status), _stream(stream)), "tq_cache_status")

    def append(self, k, v, slots, return_values: bool = False, stream=None):
        """Write rows k, v [n, kv_heads, d] (bf16 or fp32) into ``slots`` (int64
        [n], negative: skipped); with return_values, what the stored codes
        stand for, in the rows' dtype."""
        return (_calls or _load_calls()).kv4_append(self._at, self._pool, k, v, slots, return_values, stream)

    def dequant(self, slots, out_dtype=None, k=None, v=None, stream=None):
        """The rows at ``slots`` as (k, v) [n, kv_heads, d]; rows of negative slots are left as they were."""
        import torch
        _on_device(self.pool, slots, k, v)
        _want(slots, torch.int64, (slots.numel(),), "slots")
        shape, dt = (slots.numel(), self.kv_heads, self.d), out_dtype or (k.dtype if k is not None else torch.bfloat16)
        new = [x is None for x in (k, v)]
        with torch.cuda.stream(None if stream is None else torch.cuda.ExternalStream(stream.cuda_stream)):
            k = torch.zeros(shape, dtype=dt, device=slots.device) if k is None else k
            v = torch.zeros(shape, dtype=dt, device=slots.device) if v is None else v
        if stream is not None:                                # new ones belong to it, and are used on the current stream
            for x, made in zip((k, v), new):
                if made:
                    x.record_stream(torch.cuda.current_stream())
        _want(k, dt, shape, "k")
        _want(v, dt, shape, "v")
        _check(_lib.tq_kv4_dequant(self._c, _ptr(slots), shape[0], _ptr(k), _ptr(v), _dtype_code(k),
                                   _stream(stream)), "tq_kv4_dequant")
        return k, v

    def attention_workspace_bytes(self, dtype, q_heads: int, n_seqs: int, n_tokens: int, max_q: int = 1) -> int:
        import torch
        return int(_lib.tq_kv4_attention_workspace_bytes(self._c, TQ_BF16 if dtype == torch.bfloat16 else TQ_F32,
                                                         q_heads, n_seqs, n_tokens, max_q))

    def attention(self, q, page_table, seq_lens, cu_q=None, max_q: int = 1, scale: float | None = None,
                  causal: bool = True, window: int = 0, out=None, lse=None, return_lse: bool = False, workspace=None,
                  stream=None):
        """Attention of q [n_tokens, q_heads, d] over the cached tokens of
        n_seqs sequences: page_table int32 [n_seqs, max_pages], seq_lens int32
        [n_seqs], cu_q int32 [n_seqs + 1] (None: one token each); max_q: the
        largest number of new tokens of a sequence, which chooses the kernel (1
        is right for a prompt too, and slow: 2.4 ms where 0.21 do); scale
        defaults to 1/sqrt(d).  Returns out (q's shape and dtype), or (out,
        lse [n_tokens, q_heads] fp32); rows behind cu_q[-1] are not written
        (in new tensors they hold anything)."""
        return (_calls or _load_calls()).kv4_attention(self._at, self._pool, q, page_table, seq_lens, cu_q, max_q, scale,
                                                       causal, window, out, lse, return_lse, workspace, stream)


@dataclass
class PageMoves:
    """Pages whose contents are to be copied: pairs int32 [n, 2] of (from, to), -1 behind the last."""

    pairs: "object"
    n_pages: int

    def copy(self, pool, stream=None, n_layers=None):
        """Copy the pages of ``pool``: a contiguous tensor [n_pages, ...] or [n_layers, n_pages, ...] (see copy_pages)."""
        copy_pages(pool, self.pairs, self.n_pages, stream, n_layers)


def copy_pages(pool, pairs, n_pages: int, stream=None, n_layers: int | None = None):
    """Copy page pairs[i, 0] to page pairs[i, 1] of ``pool``, a contiguous
    tensor [n_pages, ...] or [n_layers, n_pages, ...] (a cache's pool, or one
    field of a packed cache with its rows grouped by pages).  ``n_layers`` says
    which (1: the first); it is needed where a shape of three or more dimensions
    reads both ways, [n_pages, n_pages, ...].  [n_pages, n_pages] is one layer."""
    (_calls or _load_calls()).copy_pages(pool, pairs, n_pages, n_layers, stream)


@_fixed("table", "lens", "refs", "status", "page_size", "n_pages")
class PageTable:
    """Which pages a cache's sequences own: table int32 [n_seqs, max_pages],
    lens int32 [n_seqs], refs int32 [n_pages], on the current CUDA device.
    Every method works in place, or leaves this table as it is and writes
    ``out`` (another PageTable of the same sizes)."""

    def __init__(self, table, lens, refs, page_size: int):
        import torch
        _on_device(table, lens, refs)
        _want(table, torch.int32, (lens.numel(), table.shape[1]), "table")
        _want(lens, torch.int32, (lens.numel(),), "lens")
        _want(refs, torch.int32, (refs.numel(),), "refs")
        self._table, self._lens, self._refs, self._page_size = table, lens, refs, page_size
        self._status = torch.zeros(1, dtype=torch.int32, device=table.device)
        self._n_pages = refs.numel()
        self._c = _Pages(table.data_ptr(), lens.data_ptr(), refs.data_ptr(), lens.numel(), table.shape[1],
                         self._n_pages, page_size, self._status.data_ptr())
        self._at = ctypes.addressof(self._c)

    @staticmethod
    def empty(n_seqs: int, max_pages: int, n_pages: int, page_size: int, device="cuda") -> "PageTable":
        import torch
        return PageTable(torch.full((n_seqs, max_pages), -1, dtype=torch.int32, device=device),
                         torch.zeros(n_seqs, dtype=torch.int32, device=device),
                         torch.zeros(n_pages, dtype=torch.int32, device=device), page_size)

    def check(self, stream=None):
        """Wait for the stream and raise what kernels recorded (a call that did nothing, and why)."""
        _on_device(self._status)                                 # another device's stream would not be the one to wait for
        _check(_lib.tq_cache_status(_ptr(self.status), _stream(stream)), "tq_cache_status")

    def extend(self, seqs, new_tokens, n_slots: int, out=None, workspace=None, stream=None):
        """Room for new_tokens[i] more tokens of sequence seqs[i] (int32 [n]
        each); returns the slots of the new tokens (int64 [n_slots], -1 behind the last)."""
        out = out or self
        return (_calls or _load_calls()).pages_extend(self._at, out._at, self._table, out.table, seqs, new_tokens, n_slots,
                                                      workspace, stream)

    def fork(self, src, dst, out=None, moves=None, workspace=None, stream=None) -> PageMoves:
        """Sequence dst[i] (empty) becomes a copy of src[i]; the moves are still to be copied."""
        out = out or self
        return PageMoves((_calls or _load_calls()).pages_fork(self._at, out._at, self._table, out.table, src, dst, moves,
                                                              workspace, stream), self.n_pages)

    def free(self, seqs, out=None, workspace=None, stream=None):
        """Sequences ``seqs`` (int32 [n]) end."""
        out = out or self
        (_calls or _load_calls()).pages_free(self._at, out._at, self._table, out.table, seqs, workspace, stream)

    def compact(self, out=None, moves=None, workspace=None, stream=None) -> PageMoves:
        """The used pages move to the front; the moves are still to be copied."""
        out = out or self
        return PageMoves((_calls or _load_calls()).pages_compact(self._at, out._at, self._table, out.table, moves, workspace,
                                                                 stream), self.n_pages)


def topk(scores, k: int, stream=None):
    import torch
    rows, cols = scores.shape
    idx = torch.empty((rows, k), dtype=torch.int32, device=scores.device)
    val = torch.empty((rows, k), dtype=torch.float32, device=scores.device)
    _check(_lib.tq_topk(_ptr(scores), rows, cols, k, _ptr(idx), _ptr(val), _stream(stream)), "tq_topk")
    return idx, val


def logits_bf16(q, keys, n_sets: int, g: int, n_keys: int, out=None, stream=None):
    """Plain bf16-key logits: q [n_sets*g, d], keys [n_sets*n_keys, d] bf16."""
    import torch
    d = q.shape[-1]
    if out is None:
        out = torch.empty((n_sets, g, n_keys), dtype=torch.float32, device=q.device)
    _check(_lib.tq_logits_bf16(_ptr(q), _ptr(keys), n_sets, g, n_keys, d, _ptr(out), _stream(stream)),
           "tq_logits_bf16")
    return out


def call_status(name: str, *args) -> int:
    """Raw call of an entry point (for API tests)."""
    return getattr(_lib, name)(*args)


def last_error() -> str:
    return _lib.tq_last_error().decode(errors="replace")
