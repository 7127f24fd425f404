// C ABI of the paged 4-bit cache, the query / key step before it and the page
// table: argument checks on the host, then the launches (include/tq.h).
#include <cuda_runtime.h>

#include <cmath>
#include <string>

#include "kv4_internal.h"
#include "tq_internal.h"

namespace {

using namespace tq;

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

tq_status cuda_fail(int err, const char* what) {
  cudaGetLastError();                          // the thread's last error goes with the report
  return fail(TQ_ERR_CUDA, std::string(what) + ": " + cuda_error_string(err));
}

bool good_d(int d) { return d == 64 || d == 128 || d == 256; }

tq_status check_sizes(int d, int kv_heads, int page_size) {
  if (!good_d(d)) return fail(TQ_ERR_INVALID_ARG, "d must be 64, 128 or 256");
  if (kv_heads < 1 || kv_heads > 1024) return fail(TQ_ERR_INVALID_ARG, "kv_heads must be in [1, 1024]");
  if (page_size < 16 || page_size > 4096 || page_size % 16)
    return fail(TQ_ERR_INVALID_ARG, "page_size must be a multiple of 16 in [16, 4096]");
  return TQ_OK;
}

tq_status check_cache(const tq_kv4& c) {
  tq_status st = check_sizes(c.d, c.kv_heads, c.page_size);
  if (st != TQ_OK) return st;
  if (c.n_pages < 1 || c.n_pages > (int64_t(1) << 30)) return fail(TQ_ERR_INVALID_ARG, "n_pages must be in [1, 2^30]");
  if (!c.pool) return fail(TQ_ERR_INVALID_ARG, "pool is NULL");
  if (!aligned(c.pool, 16)) return fail(TQ_ERR_INVALID_ARG, "pool must be 16-byte aligned");
  if (!aligned(c.status, 4)) return fail(TQ_ERR_INVALID_ARG, "status must be 4-byte aligned");
  return TQ_OK;
}

tq_status check_dtype(tq_dtype t) {
  if (t != TQ_BF16 && t != TQ_F32) return fail(TQ_ERR_INVALID_ARG, "dtype must be TQ_BF16 or TQ_F32");
  return TQ_OK;
}

// rows [n, heads * d] with a token stride: non-null, 16-byte aligned rows
tq_status check_rows(const void* p, int64_t ld, int64_t width, tq_dtype t, const char* what) {
  const int64_t esz = t == TQ_BF16 ? 2 : 4;
  if (!p) return fail(TQ_ERR_INVALID_ARG, std::string(what) + " is NULL");
  if (ld < width || ld > (int64_t(1) << 40)) return fail(TQ_ERR_INVALID_ARG, std::string(what) + ": token stride below heads * d");
  if (!aligned(p, 16) || (ld * esz) % 16)
    return fail(TQ_ERR_INVALID_ARG, std::string(what) + ": rows and row strides must be 16-byte aligned");
  return TQ_OK;
}

tq_status check_pages(const tq_pages& p, const char* what) {
  if (p.n_seqs < 1 || p.n_seqs > (int64_t(1) << 20)) return fail(TQ_ERR_INVALID_ARG, "n_seqs must be in [1, 2^20]");
  if (p.max_pages < 1 || p.max_pages > INT32_MAX) return fail(TQ_ERR_INVALID_ARG, "max_pages must be in [1, 2^31)");
  if (p.n_pages < 1 || p.n_pages > (int64_t(1) << 30)) return fail(TQ_ERR_INVALID_ARG, "n_pages must be in [1, 2^30]");
  if (p.page_size < 1) return fail(TQ_ERR_INVALID_ARG, "page_size must be >= 1");
  if (!p.table || !p.lens || !p.refs) return fail(TQ_ERR_INVALID_ARG, std::string(what) + ": an array is NULL");
  if (!aligned(p.table, 4) || !aligned(p.lens, 4) || !aligned(p.refs, 4) || !aligned(p.status, 4))
    return fail(TQ_ERR_INVALID_ARG, std::string(what) + ": arrays must be 4-byte aligned");
  return TQ_OK;
}

tq_status check_call(const tq_pages& in, const tq_pages& out, int64_t n, const void* ws, size_t ws_bytes) {
  tq_status st = check_pages(in, "in");
  if (st != TQ_OK || (st = check_pages(out, "out")) != TQ_OK) return st;
  if (in.n_seqs != out.n_seqs || in.max_pages != out.max_pages || in.n_pages != out.n_pages ||
      in.page_size != out.page_size)
    return fail(TQ_ERR_INVALID_ARG, "in and out differ in their sizes");
  const bool same = in.table == out.table;
  if ((in.lens == out.lens) != same || (in.refs == out.refs) != same)
    return fail(TQ_ERR_INVALID_ARG, "out must be in's three arrays or three others");
  if (n < 0 || n > in.n_seqs) return fail(TQ_ERR_INVALID_ARG, "n must be in [0, n_seqs]");
  if (!ws || ws_bytes < pages_ws_bytes(in, n)) return fail(TQ_ERR_INVALID_ARG, "workspace missing or too small");
  if (!aligned(ws, 16)) return fail(TQ_ERR_INVALID_ARG, "workspace must be 16-byte aligned");
  return TQ_OK;
}

}  // namespace

extern "C" {

tq_status tq_qk_norm_rope(const void* q, int64_t ld_q, int q_heads, const void* k, int64_t ld_k, int k_heads,
                          tq_dtype dtype, int64_t n_tokens, int d, const float* w_q, const float* w_k, float eps,
                          const int64_t* positions, int n_axes, int rot_dim, int interleaved, const double* inv_freq,
                          const int32_t* axis, void* out_q, int64_t ld_out_q, void* out_k, int64_t ld_out_k,
                          void* stream) {
  tq_status st = check_dtype(dtype);
  if (st != TQ_OK) return st;
  if (!good_d(d)) return fail(TQ_ERR_INVALID_ARG, "d must be 64, 128 or 256");
  if (q_heads < 0 || k_heads < 0 || q_heads > 65536 || k_heads > 65536)
    return fail(TQ_ERR_INVALID_ARG, "q_heads and k_heads must be in [0, 65536]");
  if (n_tokens < 0 || n_tokens > INT32_MAX) return fail(TQ_ERR_INVALID_ARG, "n_tokens must be in [0, 2^31)");
  if (!(eps > 0.f) || !std::isfinite(eps)) return fail(TQ_ERR_INVALID_ARG, "eps must be positive and finite");
  if (rot_dim < 0 || rot_dim > d || rot_dim % 2) return fail(TQ_ERR_INVALID_ARG, "rot_dim must be even and in [0, d]");
  if (n_axes < 1 || n_axes > 4) return fail(TQ_ERR_INVALID_ARG, "n_axes must be in [1, 4]");
  if (rot_dim && !inv_freq) return fail(TQ_ERR_INVALID_ARG, "inv_freq is NULL");
  RopeArgs a = {};
  for (int i = 0; i < rot_dim / 2; ++i) {
    if (!std::isfinite(inv_freq[i])) return fail(TQ_ERR_INVALID_ARG, "inv_freq must be finite");
    if (axis && (axis[i] < 0 || axis[i] >= n_axes)) return fail(TQ_ERR_INVALID_ARG, "axis must be in [0, n_axes)");
    a.turns[i] = inv_freq[i] / (2.0 * std::acos(-1.0));
    a.axis[i] = axis ? static_cast<uint8_t>(axis[i]) : 0;
  }
  if (n_tokens == 0 || q_heads + k_heads == 0) return TQ_OK;
  if (rot_dim && (!positions || !aligned(positions, 8)))
    return fail(TQ_ERR_INVALID_ARG, "positions is NULL or not 8-byte aligned");
  if (!aligned(w_q, 4) || !aligned(w_k, 4)) return fail(TQ_ERR_INVALID_ARG, "weights must be 4-byte aligned");
  if (q_heads) {
    if ((st = check_rows(q, ld_q, static_cast<int64_t>(q_heads) * d, dtype, "q")) != TQ_OK) return st;
    if ((st = check_rows(out_q, ld_out_q, static_cast<int64_t>(q_heads) * d, dtype, "out_q")) != TQ_OK) return st;
    if (out_q == q && ld_out_q != ld_q) return fail(TQ_ERR_INVALID_ARG, "in place, out_q needs q's token stride");
  }
  if (k_heads) {
    if ((st = check_rows(k, ld_k, static_cast<int64_t>(k_heads) * d, dtype, "k")) != TQ_OK) return st;
    if ((st = check_rows(out_k, ld_out_k, static_cast<int64_t>(k_heads) * d, dtype, "out_k")) != TQ_OK) return st;
    if (out_k == k && ld_out_k != ld_k) return fail(TQ_ERR_INVALID_ARG, "in place, out_k needs k's token stride");
  }
  a.x[0] = q; a.x[1] = k;
  a.y[0] = out_q; a.y[1] = out_k;
  a.w[0] = w_q; a.w[1] = w_k;
  a.ld_x[0] = ld_q; a.ld_x[1] = ld_k;
  a.ld_y[0] = ld_out_q; a.ld_y[1] = ld_out_k;
  a.heads[0] = q_heads; a.heads[1] = k_heads;
  a.n_tokens = n_tokens;
  a.d = d; a.rot_dim = rot_dim; a.interleaved = interleaved != 0; a.n_axes = n_axes;
  a.eps = eps;
  a.positions = positions;
  const int err = launch_qk_norm_rope(a, dtype == TQ_BF16, stream);
  return err ? cuda_fail(err, "tq_qk_norm_rope launch") : TQ_OK;
}

size_t tq_kv4_page_bytes(int d, int kv_heads, int page_size) {
  if (check_sizes(d, kv_heads, page_size) != TQ_OK) return 0;
  return static_cast<size_t>(kv_heads) * (page_size / 16) * 18 * d;
}

tq_status tq_kv4_append(tq_kv4 cache, const void* k, int64_t ld_k, const void* v, int64_t ld_v, tq_dtype dtype,
                        int64_t n_tokens, const int64_t* slots, void* k_values, void* v_values, void* stream) {
  tq_status st = check_cache(cache);
  if (st != TQ_OK || (st = check_dtype(dtype)) != TQ_OK) return st;
  if (n_tokens < 0 || n_tokens > (int64_t(1) << 24)) return fail(TQ_ERR_INVALID_ARG, "n_tokens must be in [0, 2^24]");
  if (n_tokens == 0) return TQ_OK;
  const int64_t width = static_cast<int64_t>(cache.kv_heads) * cache.d;
  if ((st = check_rows(k, ld_k, width, dtype, "k")) != TQ_OK) return st;
  if ((st = check_rows(v, ld_v, width, dtype, "v")) != TQ_OK) return st;
  if (!slots || !aligned(slots, 8)) return fail(TQ_ERR_INVALID_ARG, "slots is NULL or not 8-byte aligned");
  if ((k_values && (k_values == k || k_values == v)) || (v_values && (v_values == k || v_values == v)) ||
      (k_values && k_values == v_values))
    return fail(TQ_ERR_INVALID_ARG, "k_values and v_values must be arrays of their own");
  if (!aligned(k_values, 16) || !aligned(v_values, 16))
    return fail(TQ_ERR_INVALID_ARG, "k_values and v_values must be 16-byte aligned");
  if (take_injected_launch_failure()) return cuda_fail(cudaErrorLaunchFailure, "tq_kv4_append launch");
  const int err = launch_kv4_append(cache, k, ld_k, v, ld_v, dtype == TQ_BF16, n_tokens, slots, k_values, v_values,
                                    stream);
  return err ? cuda_fail(err, "tq_kv4_append launch") : TQ_OK;
}

tq_status tq_kv4_dequant(tq_kv4 cache, const int64_t* slots, int64_t n_tokens, void* k, void* v, tq_dtype dtype,
                         void* stream) {
  tq_status st = check_cache(cache);
  if (st != TQ_OK || (st = check_dtype(dtype)) != TQ_OK) return st;
  if (n_tokens < 0 || n_tokens > (int64_t(1) << 24)) return fail(TQ_ERR_INVALID_ARG, "n_tokens must be in [0, 2^24]");
  if (n_tokens == 0 || (!k && !v)) return TQ_OK;
  if (!slots || !aligned(slots, 8)) return fail(TQ_ERR_INVALID_ARG, "slots is NULL or not 8-byte aligned");
  if (!aligned(k, 16) || !aligned(v, 16)) return fail(TQ_ERR_INVALID_ARG, "k and v must be 16-byte aligned");
  const int err = launch_kv4_dequant(cache, slots, n_tokens, k, v, dtype == TQ_BF16, stream);
  return err ? cuda_fail(err, "tq_kv4_dequant launch") : TQ_OK;
}

size_t tq_kv4_attention_workspace_bytes(tq_kv4 cache, tq_dtype dtype, int q_heads, int64_t n_seqs, int64_t n_tokens,
                                        int max_q) {
  if (n_seqs <= 0 || n_tokens <= 0 || !good_d(cache.d) || cache.kv_heads < 1 || q_heads < 1 || max_q < 1) return 0;
  return kv4_attention_ws_bytes(cache.d, dtype == TQ_BF16, static_cast<int64_t>(max_q) * (q_heads / cache.kv_heads));
}

tq_status tq_kv4_attention(tq_kv4 cache, const void* q, tq_dtype dtype, int64_t ld_q, int q_heads, int64_t n_tokens,
                           int64_t n_seqs, const int32_t* cu_q, int max_q, const int32_t* page_table,
                           int64_t ld_table, const int32_t* seq_lens, float scale, int causal, int window, void* out,
                           float* lse, void* workspace, size_t workspace_bytes, void* stream) {
  tq_status st = check_cache(cache);
  if (st != TQ_OK || (st = check_dtype(dtype)) != TQ_OK) return st;
  if (q_heads < cache.kv_heads || q_heads % cache.kv_heads || q_heads > 65536)
    return fail(TQ_ERR_INVALID_ARG, "q_heads must be a multiple of kv_heads, at most 65536");
  if (n_tokens < 0 || n_tokens > (int64_t(1) << 24)) return fail(TQ_ERR_INVALID_ARG, "n_tokens must be in [0, 2^24]");
  if (n_seqs < 0) return fail(TQ_ERR_INVALID_ARG, "n_seqs < 0");
  if (n_seqs > 65535) return fail(TQ_ERR_UNSUPPORTED, "n_seqs must be <= 65535");
  if (!cu_q && n_tokens != n_seqs) return fail(TQ_ERR_INVALID_ARG, "without cu_q there is one token per sequence");
  if (max_q < 1) return fail(TQ_ERR_INVALID_ARG, "max_q must be >= 1");
  if (!std::isfinite(scale)) return fail(TQ_ERR_INVALID_ARG, "scale must be finite");
  if (window < 0) return fail(TQ_ERR_INVALID_ARG, "window must be >= 0");
  if (window > 0 && !causal) return fail(TQ_ERR_INVALID_ARG, "a window needs causal");
  if (n_seqs == 0 || n_tokens == 0) return TQ_OK;
  if ((st = check_rows(q, ld_q, static_cast<int64_t>(q_heads) * cache.d, dtype, "q")) != TQ_OK) return st;
  if (!out || !aligned(out, 16)) return fail(TQ_ERR_INVALID_ARG, "out is NULL or not 16-byte aligned");
  if (!page_table || !seq_lens) return fail(TQ_ERR_INVALID_ARG, "page_table or seq_lens is NULL");
  if (ld_table < 1 || ld_table > INT32_MAX) return fail(TQ_ERR_INVALID_ARG, "ld_table must be in [1, 2^31)");
  if (!aligned(page_table, 4) || !aligned(seq_lens, 4) || !aligned(cu_q, 4) || !aligned(lse, 4))
    return fail(TQ_ERR_INVALID_ARG, "page_table, seq_lens, cu_q and lse must be 4-byte aligned");
  const size_t need = tq_kv4_attention_workspace_bytes(cache, dtype, q_heads, n_seqs, n_tokens, max_q);
  if (!workspace || workspace_bytes < need) return fail(TQ_ERR_INVALID_ARG, "workspace missing or too small");
  if (!aligned(workspace, 16)) return fail(TQ_ERR_INVALID_ARG, "workspace must be 16-byte aligned");
  Kv4Attn a;
  a.c = cache;
  a.q = q;
  a.ld_q = ld_q;
  a.n_tokens = n_tokens;
  a.ld_table = ld_table;
  a.q_heads = q_heads;
  a.n_seqs = static_cast<int>(n_seqs);
  a.max_q = max_q;
  a.cu_q = cu_q;
  a.page_table = page_table;
  a.seq_lens = seq_lens;
  a.scale = scale;
  a.causal = causal != 0;
  a.window = window;
  a.out = out;
  a.lse = lse;
  a.ws = workspace;
  const int err = launch_kv4_attention(a, dtype == TQ_BF16, stream);
  return err ? cuda_fail(err, "tq_kv4_attention launch") : TQ_OK;
}

size_t tq_pages_workspace_bytes(tq_pages pages, int64_t n) {
  if (pages.n_seqs < 1 || pages.n_pages < 1 || n < 0) return 0;
  return pages_ws_bytes(pages, n);
}

tq_status tq_pages_extend(tq_pages in, tq_pages out, int64_t n, const int32_t* seqs, const int32_t* new_tokens,
                          int64_t* slots, int64_t n_slots, void* workspace, size_t workspace_bytes, void* stream) {
  tq_status st = check_call(in, out, n, workspace, workspace_bytes);
  if (st != TQ_OK) return st;
  if (n && (!seqs || !new_tokens || !aligned(seqs, 4) || !aligned(new_tokens, 4)))
    return fail(TQ_ERR_INVALID_ARG, "seqs and new_tokens must be given, 4-byte aligned");
  if (n_slots < 0 || n_slots > INT32_MAX || !aligned(slots, 8))   // the new tokens' places in the list are 32-bit numbers
    return fail(TQ_ERR_INVALID_ARG, "n_slots must be in [0, 2^31), slots 8-byte aligned");
  const int err = launch_pages_extend(in, out, n, seqs, new_tokens, slots, n_slots, workspace, stream);
  return err ? cuda_fail(err, "tq_pages_extend launch") : TQ_OK;
}

tq_status tq_pages_fork(tq_pages in, tq_pages out, int64_t n, const int32_t* src, const int32_t* dst, int32_t* moves,
                        void* workspace, size_t workspace_bytes, void* stream) {
  tq_status st = check_call(in, out, n, workspace, workspace_bytes);
  if (st != TQ_OK) return st;
  if (n && (!src || !dst || !moves || !aligned(src, 4) || !aligned(dst, 4) || !aligned(moves, 4)))
    return fail(TQ_ERR_INVALID_ARG, "src, dst and moves must be given, 4-byte aligned");
  const int err = launch_pages_fork(in, out, n, src, dst, moves, workspace, stream);
  return err ? cuda_fail(err, "tq_pages_fork launch") : TQ_OK;
}

tq_status tq_pages_free(tq_pages in, tq_pages out, int64_t n, const int32_t* seqs, void* workspace,
                        size_t workspace_bytes, void* stream) {
  // a list may name a sequence twice: only its length is bounded
  tq_status st = check_call(in, out, 0, workspace, workspace_bytes);
  if (st != TQ_OK) return st;
  if (n < 0 || n > INT32_MAX) return fail(TQ_ERR_INVALID_ARG, "n must be in [0, 2^31)");
  if (workspace_bytes < pages_ws_bytes(in, n)) return fail(TQ_ERR_INVALID_ARG, "workspace missing or too small");
  if (n && (!seqs || !aligned(seqs, 4))) return fail(TQ_ERR_INVALID_ARG, "seqs must be given, 4-byte aligned");
  const int err = launch_pages_free(in, out, n, seqs, workspace, stream);
  return err ? cuda_fail(err, "tq_pages_free launch") : TQ_OK;
}

tq_status tq_pages_compact(tq_pages in, tq_pages out, int32_t* moves, void* workspace, size_t workspace_bytes,
                           void* stream) {
  tq_status st = check_call(in, out, 0, workspace, workspace_bytes);
  if (st != TQ_OK) return st;
  if (!moves || !aligned(moves, 4)) return fail(TQ_ERR_INVALID_ARG, "moves must be given, 4-byte aligned");
  const int err = launch_pages_compact(in, out, moves, workspace, stream);
  return err ? cuda_fail(err, "tq_pages_compact launch") : TQ_OK;
}

tq_status tq_pages_copy(void* base, int64_t n_layers, int64_t layer_stride, int64_t page_bytes, int64_t n_pages,
                        const int32_t* moves, int64_t n_moves, void* stream) {
  if (n_layers < 0 || n_layers > 65536 || n_moves < 0 || n_moves > (int64_t(1) << 30))
    return fail(TQ_ERR_INVALID_ARG, "n_layers must be in [0, 65536] and n_moves in [0, 2^30]");
  if (n_pages < 1 || n_pages > (int64_t(1) << 30)) return fail(TQ_ERR_INVALID_ARG, "n_pages must be in [1, 2^30]");
  if (page_bytes < 4 || page_bytes % 4 || page_bytes > (int64_t(1) << 32) || layer_stride % 4)
    return fail(TQ_ERR_INVALID_ARG, "page_bytes and layer_stride must be multiples of 4, page_bytes in [4, 2^32]");
  if (n_layers > 1 && layer_stride < page_bytes * n_pages)
    return fail(TQ_ERR_INVALID_ARG, "layer_stride is less than a layer's pages");
  if (n_layers == 0 || n_moves == 0) return TQ_OK;
  if (!base || !aligned(base, 4)) return fail(TQ_ERR_INVALID_ARG, "base is NULL or not 4-byte aligned");
  if (!moves || !aligned(moves, 4)) return fail(TQ_ERR_INVALID_ARG, "moves is NULL or not 4-byte aligned");
  const int err = launch_pages_copy(base, n_layers, layer_stride, page_bytes, n_pages, moves, n_moves, stream);
  return err ? cuda_fail(err, "tq_pages_copy launch") : TQ_OK;
}

tq_status tq_cache_status(int32_t* status, void* stream) {
  if (!status || !aligned(status, 4)) return fail(TQ_ERR_INVALID_ARG, "status is NULL or not 4-byte aligned");
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  int32_t bits = 0;
  cudaError_t e = cudaMemcpyAsync(&bits, status, sizeof(bits), cudaMemcpyDeviceToHost, st);
  if (e == cudaSuccess) e = cudaMemsetAsync(status, 0, sizeof(bits), st);
  if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  if (e != cudaSuccess) return cuda_fail(e, "tq_cache_status");
  if (bits & kStatusWait) return fail(TQ_ERR_CUDA, "a bounded wait ran out in a kernel");
  if (bits & kStatusIndex) return fail(TQ_ERR_INVALID_ARG, "an index was out of range, or a sequence not as the call needs it");
  if (bits & kStatusPages) return fail(TQ_ERR_INVALID_ARG, "a page, length or token range was out of range");
  if (bits & kStatusNoPages) return fail(TQ_ERR_NOMEM, "too few free pages");
  return bits ? fail(TQ_ERR_CUDA, "unknown status bits") : TQ_OK;
}

}  // extern "C"
