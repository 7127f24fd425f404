// The calls that a decode step makes for every layer, from Python in one step:
// checks of the tensors, outputs and workspaces, and the C ABI's entry point.
// The same in Python over ctypes took more of the host than the kernels of a
// small batch take of the GPU (one token: norm and rotation 13.9 us against 2.2
// on the GPU; append of 64 tokens 10.6 against 3.0; attention over 1000 tokens
// 17.6 against 12); here these calls take 6.4, 5.8 and 11 us.
//
// libtq is not linked: tq.py hands over the addresses of its entry points
// (bind), so that there is one copy of it, the one that ctypes loaded.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <cmath>
#include <optional>
#include <stdexcept>
#include <string>

#include "../../../include/tq.h"

namespace {

// ------------------------------------------------------- libtq and errors --

struct Entry {
  decltype(&tq_qk_norm_rope) qk_norm_rope;
  decltype(&tq_kv4_append) kv4_append;
  decltype(&tq_kv4_attention) kv4_attention;
  decltype(&tq_kv4_attention_workspace_bytes) kv4_attention_workspace_bytes;
  decltype(&tq_pages_workspace_bytes) pages_workspace_bytes;
  decltype(&tq_pages_extend) pages_extend;
  decltype(&tq_pages_fork) pages_fork;
  decltype(&tq_pages_free) pages_free;
  decltype(&tq_pages_compact) pages_compact;
  decltype(&tq_pages_copy) pages_copy;
} tqlib = {};
PyObject* raise_status = nullptr;              // tq._check: raises TQError(status, name)

struct ValueError : std::runtime_error { using runtime_error::runtime_error; };
struct TypeError : std::runtime_error { using runtime_error::runtime_error; };
struct Raised {};                              // a Python error is set already

void check(tq_status st, const char* where) {
  if (st == TQ_OK) return;
  PyObject* r = PyObject_CallFunction(raise_status, "is", static_cast<int>(st), where);
  Py_XDECREF(r);
  throw Raised();
}

template <typename F>
PyObject* guarded(F f) {
  try {
    return f();
  } catch (const Raised&) {
  } catch (const ValueError& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const TypeError& e) {
    PyErr_SetString(PyExc_TypeError, e.what());
  } catch (...) {                              // torch's own, out of device memory among them
    torch::translate_exception_to_python(std::current_exception());
  }
  return nullptr;
}

// Others run while memory is found and kernels are launched, as in torch's own
// calls: a full launch queue may wait for one of them.
struct NoGil {
  PyThreadState* state = PyEval_SaveThread();
  NoGil() = default;
  NoGil(const NoGil&) = delete;
  ~NoGil() { PyEval_RestoreThread(state); }
};

// -------------------------------------------------------------- arguments --

long long integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Raised();
  return v;
}
int small(PyObject* o, const char* what) {
  const long long v = integer(o);
  if (v < INT32_MIN || v > INT32_MAX) throw ValueError(std::string(what) + " is out of range");
  return static_cast<int>(v);
}
double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Raised();
  return v;
}
bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Raised();
  return v != 0;
}
template <typename T>
const T* address(PyObject* o) { return reinterpret_cast<const T*>(static_cast<uintptr_t>(integer(o))); }

// A tensor argument; None is an undefined one.
at::Tensor tensor(PyObject* o, const char* what, bool needed = true) {
  if (o == Py_None && !needed) return {};
  if (!THPVariable_Check(o)) throw TypeError(std::string(what) + " must be a tensor");
  return THPVariable_Unpack(o);
}
void* ptr(const at::Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }
const int32_t* ids(const at::Tensor& t) { return static_cast<const int32_t*>(ptr(t)); }

// The current device, on which every tensor has to be, and the stream of the
// call: `stream` or the device's current one.  Outputs and workspaces belong to
// that stream, so that the memory of a workspace that goes is not given to
// another stream's work while the kernel runs; outputs are also known to be used
// on the current one.
struct Place {
  c10::DeviceIndex dev;
  void* stream;
  std::optional<c10::cuda::CUDAStream> cur;
  std::optional<c10::cuda::CUDAStreamGuard> guard;
  explicit Place(PyObject* s) : dev(c10::cuda::current_device()) {
    if (s == Py_None) {
      stream = c10::cuda::getCurrentCUDAStream(dev).stream();
      return;
    }
    PyObject* raw = PyObject_GetAttrString(s, "cuda_stream");
    if (!raw) throw Raised();
    const unsigned long long v = PyLong_AsUnsignedLongLong(raw);
    Py_DECREF(raw);
    if (PyErr_Occurred()) throw Raised();
    stream = reinterpret_cast<void*>(static_cast<uintptr_t>(v));
    cur = c10::cuda::getCurrentCUDAStream(dev);
    if (cur->stream() != stream)
      guard.emplace(c10::cuda::getStreamFromExternal(static_cast<cudaStream_t>(stream), dev));
  }
  at::Tensor output(at::Tensor t) const {
    if (guard) c10::cuda::CUDACachingAllocator::recordStream(t.storage().data_ptr(), *cur);
    return t;
  }
  void on(const at::Tensor& t) const {
    if (t.defined() && (!t.is_cuda() || t.get_device() != dev))
      throw ValueError("a tensor is on " + t.device().str() + ", the current device is cuda:" + std::to_string(dev));
  }
  template <typename... Ts>
  void all(const Ts&... ts) const { (on(ts), ...); }
};

tq_dtype dtype(const at::Tensor& t) {
  if (t.scalar_type() == at::kBFloat16) return TQ_BF16;
  if (t.scalar_type() == at::kFloat) return TQ_F32;
  throw TypeError(std::string("unsupported dtype ") + c10::toString(t.scalar_type()));
}

// A [tokens, heads, d] tensor whose heads are contiguous: its token stride.
int64_t token_stride(const at::Tensor& x, const char* what) {
  if (x.dim() != 3) throw ValueError(std::string(what) + " must be [tokens, heads, d] with contiguous heads");
  const int64_t n = x.size(0), h = x.size(1), d = x.size(2);
  if (x.numel() && (x.stride(2) != 1 || (h > 1 && x.stride(1) != d)))
    throw ValueError(std::string(what) + " must be [tokens, heads, d] with contiguous heads");
  return n > 1 ? x.stride(0) : h * d;          // of a single token torch keeps any stride
}

void want(const at::Tensor& x, at::ScalarType t, at::IntArrayRef shape, const char* what) {
  if (!x.defined() || (x.scalar_type() == t && x.sizes() == shape && x.is_contiguous())) return;
  std::string s;
  for (const int64_t v : shape) s += (s.empty() ? "" : ", ") + std::to_string(v);
  throw ValueError(std::string(what) + " must be contiguous " + c10::toString(t) + " of shape (" + s + ")");
}

at::Tensor make(const at::Tensor& like, at::IntArrayRef shape) { return at::empty(shape, like.options()); }
at::Tensor make(const at::Tensor& like, at::IntArrayRef shape, at::ScalarType t) {
  return at::empty(shape, like.options().dtype(t));
}
// `given`, or a new one of `need` bytes; its bytes
at::Tensor workspace(const at::Tensor& given, size_t need, const at::Tensor& like, size_t* bytes) {
  if (given.defined() && !given.is_contiguous()) throw ValueError("workspace must be contiguous");   // its bytes are its own
  at::Tensor w = given.defined() ? given : make(like, {static_cast<int64_t>(need)}, at::kByte);
  *bytes = w.nbytes();
  return w;
}

void count(Py_ssize_t n, Py_ssize_t want) {
  if (n != want) throw TypeError("wrong number of arguments");
  if (!raise_status) throw TypeError("libtq's entry points are not bound");
}

PyObject* pair(at::Tensor a, at::Tensor b) {
  PyObject *x = THPVariable_Wrap(std::move(a)), *y = THPVariable_Wrap(std::move(b));
  PyObject* t = x && y ? PyTuple_Pack(2, x, y) : nullptr;
  Py_XDECREF(x);
  Py_XDECREF(y);
  return t;
}

// ------------------------------------------------------------------ calls --

// q, k, positions, (rot_dim, interleaved, inv_freq, axis), q_weight, k_weight, eps, out_q, out_k, stream
PyObject* qk_norm_rope(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  return guarded([&]() -> PyObject* {
    count(n_args, 10);
    const at::Tensor q = tensor(a[0], "q"), k = tensor(a[1], "k"), pos = tensor(a[2], "positions");
    const at::Tensor wq = tensor(a[4], "q_weight", false), wk = tensor(a[5], "k_weight", false);
    at::Tensor oq = tensor(a[7], "out_q", false), ok = tensor(a[8], "out_k", false);
    Place at(a[9]);
    at.all(q, k, pos, wq, wk, oq, ok);
    const int64_t ld_q = token_stride(q, "q"), ld_k = token_stride(k, "k");
    const int64_t n = q.size(0), d = q.size(2);
    if (k.size(0) != n || k.size(2) != d || k.scalar_type() != q.scalar_type())
      throw ValueError("q and k must agree in tokens, d and dtype");
    const int64_t axes = pos.dim() == 2 ? pos.size(0) : 1;
    if (pos.dim() == 2) want(pos, at::kLong, {axes, n}, "positions");
    else want(pos, at::kLong, {n}, "positions");
    want(wq, at::kFloat, {d}, "q_weight");
    want(wk, at::kFloat, {d}, "k_weight");
    const tq_dtype t = dtype(q);
    if (!PyTuple_Check(a[3]) || PyTuple_GET_SIZE(a[3]) != 4) throw TypeError("rope must be a plan");
    const int rot = small(PyTuple_GET_ITEM(a[3], 0), "rot_dim"), inter = small(PyTuple_GET_ITEM(a[3], 1), "interleaved");
    const double* inv_freq = address<double>(PyTuple_GET_ITEM(a[3], 2));
    const int32_t* axis = address<int32_t>(PyTuple_GET_ITEM(a[3], 3));
    const float eps = static_cast<float>(number(a[6]));
    if (axes > INT32_MAX) throw ValueError("positions has too many rows");
    std::optional<NoGil> free(std::in_place);
    if (!oq.defined()) oq = at.output(make(q, q.sizes()));
    if (!ok.defined()) ok = at.output(make(k, k.sizes()));
    if (oq.sizes() != q.sizes() || ok.sizes() != k.sizes() || oq.scalar_type() != q.scalar_type() ||
        ok.scalar_type() != q.scalar_type())
      throw ValueError("out_q and out_k must have the shapes and dtype of q and k");
    const int64_t ld_oq = token_stride(oq, "out_q"), ld_ok = token_stride(ok, "out_k");
    const tq_status st = tqlib.qk_norm_rope(
        ptr(q), ld_q, static_cast<int>(q.size(1)), ptr(k), ld_k, static_cast<int>(k.size(1)), t, n, static_cast<int>(d),
        static_cast<const float*>(ptr(wq)), static_cast<const float*>(ptr(wk)), eps, static_cast<const int64_t*>(ptr(pos)),
        static_cast<int>(axes), rot, inter, inv_freq, axis, ptr(oq), ld_oq, ptr(ok), ld_ok, at.stream);
    free.reset();
    check(st, "tq_qk_norm_rope");
    return pair(oq, ok);
  });
}

// cache, pool, k, v, slots, return_values, stream
PyObject* kv4_append(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  return guarded([&]() -> PyObject* {
    count(n_args, 7);
    const tq_kv4& c = *address<tq_kv4>(a[0]);
    const at::Tensor pool = tensor(a[1], "pool"), k = tensor(a[2], "k"), v = tensor(a[3], "v"), slots = tensor(a[4], "slots");
    Place at(a[6]);
    at.all(pool, k, v, slots);
    const int64_t shape[3] = {k.dim() == 3 ? k.size(0) : -1, c.kv_heads, c.d};
    if (k.sizes() != at::IntArrayRef(shape) || v.sizes() != at::IntArrayRef(shape) || k.scalar_type() != v.scalar_type())
      throw ValueError("k and v must both be [n, " + std::to_string(c.kv_heads) + ", " + std::to_string(c.d) + "], of one dtype");
    want(slots, at::kLong, {shape[0]}, "slots");
    const tq_dtype t = dtype(k);
    at::Tensor kv, vv;
    const bool with_values = truth(a[5]);
    const int64_t ld_k = token_stride(k, "k"), ld_v = token_stride(v, "v");
    std::optional<NoGil> free(std::in_place);
    if (with_values) {
      kv = at.output(make(k, shape));
      vv = at.output(make(k, shape));
    }
    const tq_status st = tqlib.kv4_append(c, ptr(k), ld_k, ptr(v), ld_v, t, shape[0],
                                          static_cast<const int64_t*>(ptr(slots)), ptr(kv), ptr(vv), at.stream);
    free.reset();
    check(st, "tq_kv4_append");
    if (!kv.defined()) Py_RETURN_NONE;
    return pair(kv, vv);
  });
}

// cache, pool, q, page_table, seq_lens, cu_q, max_q, scale, causal, window, out, lse, return_lse, workspace, stream
PyObject* kv4_attention(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  return guarded([&]() -> PyObject* {
    count(n_args, 15);
    const tq_kv4& c = *address<tq_kv4>(a[0]);
    const at::Tensor pool = tensor(a[1], "pool"), q = tensor(a[2], "q"), table = tensor(a[3], "page_table");
    const at::Tensor lens = tensor(a[4], "seq_lens"), cu = tensor(a[5], "cu_q", false), given = tensor(a[13], "workspace", false);
    at::Tensor out = tensor(a[10], "out", false), lse = tensor(a[11], "lse", false);
    Place at(a[14]);
    at.all(pool, q, table, lens, cu, out, lse, given);
    const int64_t ld = token_stride(q, "q"), n = q.size(0), hq = q.size(1), S = lens.numel();
    if (q.size(2) != c.d) throw ValueError("q must have d = " + std::to_string(c.d));
    want(lens, at::kInt, {S}, "seq_lens");
    want(cu, at::kInt, {S + 1}, "cu_q");
    if (table.dim() != 2) throw ValueError("page_table must be contiguous int32 [n_seqs, max_pages]");
    want(table, at::kInt, {S, table.size(1)}, "page_table");
    want(out, q.scalar_type(), q.sizes(), "out");
    want(lse, at::kFloat, {n, hq}, "lse");
    const tq_dtype t = dtype(q);
    const bool with_lse = truth(a[12]);
    const int max_q = small(a[6], "max_q");
    if (hq > 65536) throw ValueError("q has too many heads");
    const double scale = a[7] == Py_None ? 1.0 / std::sqrt(static_cast<double>(c.d)) : number(a[7]);
    const bool causal = truth(a[8]);
    const int window = small(a[9], "window");
    std::optional<NoGil> free(std::in_place);
    if (!out.defined()) out = at.output(make(q, q.sizes()));
    if (with_lse && !lse.defined()) lse = at.output(make(q, {n, hq}, at::kFloat));
    size_t bytes = 0;
    const at::Tensor ws = workspace(
        given, tqlib.kv4_attention_workspace_bytes(c, t, static_cast<int>(hq), S, n, max_q), q, &bytes);
    const tq_status st = tqlib.kv4_attention(
        c, ptr(q), t, ld, static_cast<int>(hq), n, S, ids(cu), max_q, ids(table), table.size(1), ids(lens),
        static_cast<float>(scale), causal, window, ptr(out), static_cast<float*>(ptr(lse)), ptr(ws), bytes, at.stream);
    free.reset();
    check(st, "tq_kv4_attention");
    if (!with_lse) return THPVariable_Wrap(out);
    return pair(out, lse);
  });
}

// Lists of sequences: int32, contiguous, of one length.
int64_t lists(const Place& at, const at::Tensor& x, const at::Tensor& y = {}) {
  at.all(x, y);
  const int64_t n = x.numel();
  want(x, at::kInt, {n}, "an index list");
  want(y, at::kInt, {n}, "an index list");
  return n;
}

// in, out, in's table, out's, seqs, new_tokens, n_slots, workspace, stream
PyObject* pages_extend(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  return guarded([&]() -> PyObject* {
    count(n_args, 9);
    const tq_pages &in = *address<tq_pages>(a[0]), &out = *address<tq_pages>(a[1]);
    const at::Tensor table = tensor(a[2], "table"), into = tensor(a[3], "out.table");
    const at::Tensor seqs = tensor(a[4], "seqs"), more = tensor(a[5], "new_tokens"), given = tensor(a[7], "workspace", false);
    Place at(a[8]);
    at.all(table, into, given);
    const int64_t n = lists(at, seqs, more), n_slots = integer(a[6]);
    if (n_slots < 0 || n_slots > INT32_MAX) throw ValueError("n_slots must be in [0, 2^31)");
    std::optional<NoGil> free(std::in_place);
    // a list of no slots has an address too: without one the call would take it that no list is wanted
    at::Tensor slots = at.output(make(table, {std::max<int64_t>(1, n_slots)}, at::kLong));
    size_t bytes = 0;
    const at::Tensor ws = workspace(given, tqlib.pages_workspace_bytes(in, n), table, &bytes);
    const tq_status st = tqlib.pages_extend(in, out, n, ids(seqs), ids(more), static_cast<int64_t*>(ptr(slots)), n_slots, ptr(ws), bytes,
                             at.stream);
    free.reset();
    check(st, "tq_pages_extend");
    return THPVariable_Wrap(n_slots ? slots : slots.narrow(0, 0, 0));
  });
}

// in, out, in's table, out's, src, dst, moves, workspace, stream
PyObject* pages_fork(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  return guarded([&]() -> PyObject* {
    count(n_args, 9);
    const tq_pages &in = *address<tq_pages>(a[0]), &out = *address<tq_pages>(a[1]);
    const at::Tensor table = tensor(a[2], "table"), into = tensor(a[3], "out.table");
    const at::Tensor src = tensor(a[4], "src"), dst = tensor(a[5], "dst"), given = tensor(a[7], "workspace", false);
    at::Tensor moves = tensor(a[6], "moves", false);
    Place at(a[8]);
    at.all(table, into, given, moves);
    const int64_t n = lists(at, src, dst);
    want(moves, at::kInt, {n, 2}, "moves");
    std::optional<NoGil> free(std::in_place);
    if (!moves.defined()) moves = at.output(make(table, {n, 2}));
    size_t bytes = 0;
    const at::Tensor ws = workspace(given, tqlib.pages_workspace_bytes(in, n), table, &bytes);
    const tq_status st = tqlib.pages_fork(in, out, n, ids(src), ids(dst), static_cast<int32_t*>(ptr(moves)), ptr(ws), bytes, at.stream);
    free.reset();
    check(st, "tq_pages_fork");
    return THPVariable_Wrap(moves);
  });
}

// in, out, in's table, out's, seqs, workspace, stream
PyObject* pages_free(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  return guarded([&]() -> PyObject* {
    count(n_args, 7);
    const tq_pages &in = *address<tq_pages>(a[0]), &out = *address<tq_pages>(a[1]);
    const at::Tensor table = tensor(a[2], "table"), into = tensor(a[3], "out.table");
    const at::Tensor seqs = tensor(a[4], "seqs"), given = tensor(a[5], "workspace", false);
    Place at(a[6]);
    at.all(table, into, given);
    const int64_t n = lists(at, seqs);
    std::optional<NoGil> free(std::in_place);
    size_t bytes = 0;
    const at::Tensor ws = workspace(given, tqlib.pages_workspace_bytes(in, n), table, &bytes);
    const tq_status st = tqlib.pages_free(in, out, n, ids(seqs), ptr(ws), bytes, at.stream);
    free.reset();
    check(st, "tq_pages_free");
    Py_RETURN_NONE;
  });
}

// in, out, in's table, out's, moves, workspace, stream
PyObject* pages_compact(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  return guarded([&]() -> PyObject* {
    count(n_args, 7);
    const tq_pages &in = *address<tq_pages>(a[0]), &out = *address<tq_pages>(a[1]);
    const at::Tensor table = tensor(a[2], "table"), into = tensor(a[3], "out.table"), given = tensor(a[5], "workspace", false);
    at::Tensor moves = tensor(a[4], "moves", false);
    Place at(a[6]);
    at.all(table, into, given, moves);
    const int64_t most = std::max<int64_t>(1, in.n_pages / 2);
    want(moves, at::kInt, {most, 2}, "moves");
    std::optional<NoGil> free(std::in_place);
    if (!moves.defined()) moves = at.output(make(table, {most, 2}));
    size_t bytes = 0;
    const at::Tensor ws = workspace(given, tqlib.pages_workspace_bytes(in, 0), table, &bytes);
    const tq_status st = tqlib.pages_compact(in, out, static_cast<int32_t*>(ptr(moves)), ptr(ws), bytes, at.stream);
    free.reset();
    check(st, "tq_pages_compact");
    return THPVariable_Wrap(moves);
  });
}

// pool, pairs, n_pages, n_layers, stream
PyObject* copy_pages(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  return guarded([&]() -> PyObject* {
    count(n_args, 5);
    const at::Tensor pool = tensor(a[0], "pool"), pairs = tensor(a[1], "pairs");
    const int64_t n_pages = integer(a[2]), asked = a[3] == Py_None ? -1 : integer(a[3]);
    Place at(a[4]);
    at.all(pool, pairs);
    if (pairs.dim() != 2) throw ValueError("pairs must be contiguous int32 [n, 2]");
    want(pairs, at::kInt, {pairs.size(0), 2}, "pairs");
    if (!pool.is_contiguous()) throw ValueError("pool must be contiguous");
    if (n_pages < 1) throw ValueError("n_pages must be >= 1");
    if (a[3] != Py_None && asked < 1) throw ValueError("n_layers must be >= 1");
    const bool one = pool.dim() >= 1 && pool.size(0) == n_pages && asked <= 1;
    const bool many = pool.dim() >= 2 && pool.size(1) == n_pages && (asked < 0 || pool.size(0) == asked);
    if (asked < 0 && one && many && pool.dim() >= 3 && n_pages > 1)
      throw ValueError("pool is one layer of pages or " + std::to_string(n_pages) + " layers of them: n_layers has to say which");
    if (!one && !many)
      throw ValueError("pool must be [" + std::to_string(n_pages) + ", ...] or [n_layers, " + std::to_string(n_pages) + ", ...]");
    const int64_t layers = one ? 1 : pool.size(0);
    std::optional<NoGil> free(std::in_place);
    const int64_t stride = static_cast<int64_t>(pool.nbytes()) / std::max<int64_t>(1, layers);
    const tq_status st = tqlib.pages_copy(ptr(pool), layers, stride, stride / n_pages, n_pages, ids(pairs), pairs.size(0), at.stream);
    free.reset();
    check(st, "tq_pages_copy");
    Py_RETURN_NONE;
  });
}

// The addresses of libtq's entry points by name, and the function that raises a status.
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  return guarded([&]() -> PyObject* {
    if (n_args != 2) throw TypeError("wrong number of arguments");
    auto get = [&](const char* name) {
      PyObject* v = PyDict_Check(a[0]) ? PyDict_GetItemString(a[0], name) : nullptr;
      if (!v) throw ValueError(std::string("no address of ") + name);
      return reinterpret_cast<void*>(static_cast<uintptr_t>(integer(v)));
    };
    Entry e;
#define TQ_GET(x) e.x = reinterpret_cast<decltype(e.x)>(get("tq_" #x))
    TQ_GET(qk_norm_rope);
    TQ_GET(kv4_append);
    TQ_GET(kv4_attention);
    TQ_GET(kv4_attention_workspace_bytes);
    TQ_GET(pages_workspace_bytes);
    TQ_GET(pages_extend);
    TQ_GET(pages_fork);
    TQ_GET(pages_free);
    TQ_GET(pages_compact);
    TQ_GET(pages_copy);
#undef TQ_GET
    tqlib = e;
    Py_INCREF(a[1]);
    Py_XDECREF(raise_status);
    raise_status = a[1];
    Py_RETURN_NONE;
  });
}

#define TQ_METHOD(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {TQ_METHOD(bind),         TQ_METHOD(qk_norm_rope), TQ_METHOD(kv4_append), TQ_METHOD(kv4_attention),
                         TQ_METHOD(pages_extend), TQ_METHOD(pages_fork),   TQ_METHOD(pages_free), TQ_METHOD(pages_compact),
                         TQ_METHOD(copy_pages),   {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", "Calls of libtq on tensors (see tq.py).", -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__calls() { return PyModule_Create(&module); }
