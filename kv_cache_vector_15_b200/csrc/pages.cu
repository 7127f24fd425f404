// The page table of a cache: growth, forks, ends, compaction, and the copies
// of pages that these ask for.
//
// Each table call is two kernels.  The plan (one CTA; the other CTAs of its
// grid check the entries of the rows that the call goes by, and copy `in` to
// `out` where these differ) checks every index and finds the
// free pages in order of their index; the second kernel takes a row of the
// table per CTA, and leaves all as it was if a check failed.  Ranks come from
// ballots and a scan over the CTA's warps, not from atomics, so pages are
// given out in the same order every time.  Bound: launch latency and one pass
// over refs (up to 16384 pages per step of the plan's CTA); the copies are bound by
// their bytes, 2 per byte of a moved page.  Into another table, on the GPU: 32
// sequences of 128 pages among 16384 grow by one token in 9.8 us, are freed in
// 4.8 (3.3 without the check of their rows), forked in 14.1, 16384 pages are
// planned for compaction in 15.8; 262144 pages 12.4, 9.1, 20.8 and 208.
#include <cuda_runtime.h>

#include <algorithm>

#include "kv4_internal.h"
#include "launch.cuh"
#include "tq_internal.h"

namespace tq {
namespace {

constexpr int kPlan = 1024;                    // threads of a planning CTA
constexpr int kSub = 16;                       // pages per lane and step of a pass over refs
constexpr int kRowThreads = 128;

constexpr int kOthers = 147;                   // CTAs behind the planning one, at most

// Workspace (int32 words): [0] failed, [1] used pages, [2] tokens of an
// extension, from [8] on a word per checking CTA, not 0 where it met a bad
// row; then map [n_seqs], three arrays [n], and list [n_pages].
constexpr int kHead = 160;
static_assert(8 + kOthers <= kHead && kOthers <= 2 * kRowThreads, "a word per checking CTA; a row's CTA reads them in two steps");
struct Ws {
  int32_t *head, *map, *len, *off, *tok, *list;
};
__host__ __device__ __forceinline__ Ws ws_of(void* ws, int64_t n_seqs, int64_t n) {
  int32_t *p = static_cast<int32_t*>(ws), *a = p + kHead + n_seqs;
  return {p, p + kHead, a, a + n, a + 2 * n, a + 3 * n};
}

// Exclusive sum over the CTA of one value per thread, and the total.
template <typename I>
__device__ __forceinline__ I cta_scan(I x, I* warp_sums, I* total) {
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  I y = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const I z = __shfl_up_sync(0xffffffffu, y, o);
    if (lane >= o) y += z;
  }
  __syncthreads();                             // warp_sums of a scan before this one are read
  if (lane == 31) warp_sums[warp] = y;
  __syncthreads();
  I before = 0, all = 0;
  const int warps = blockDim.x / 32;
  for (int i = 0; i < warps; ++i) {
    const I w = warp_sums[i];
    if (i < warp) before += w;
    all += w;
  }
  *total = all;
  return before + y - x;
}

// For every page in order: f(page, used, rank among the used, rank among the
// free), until `enough` free pages have gone by; the used pages seen.  One SM
// works here, so a step is no longer than the pages ask for: 1024 of them per
// place of a lane, and a search for a few free ones first looks at 4096.
template <typename F>
__device__ __forceinline__ int over_pages(const int32_t* refs, int n_pages, int enough, int* warp_sums, F f) {
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  int used_before = 0;
  for (int base = 0; base < n_pages;) {
    const int places = min(base == 0 && enough < n_pages ? 4 : kSub, (n_pages - base + kPlan - 1) / kPlan);
    const int first = base + warp * 32 * places + lane;
    uint32_t ballots[kSub];
    bool used[kSub];
    int mine = 0;
#pragma unroll
    for (int i = 0; i < kSub; ++i) {
      used[i] = false;
      if (i < places && first + 32 * i < n_pages) used[i] = refs[first + 32 * i] > 0;
    }
#pragma unroll
    for (int i = 0; i < kSub; ++i)
      if (i < places) {                        // the same for every warp
        ballots[i] = __ballot_sync(0xffffffffu, used[i]);
        mine += __popc(ballots[i]);
      }
    int all;
    // one value per warp: its first lane brings it, the others 0
    int rank = used_before + __shfl_sync(0xffffffffu, cta_scan(lane == 0 ? mine : 0, warp_sums, &all), 0);
#pragma unroll
    for (int i = 0; i < kSub; ++i)
      if (i < places) {
        const int page = first + 32 * i, u = rank + __popc(ballots[i] & ((1u << lane) - 1u));
        if (page < n_pages) f(page, used[i], u, page - u);
        rank += __popc(ballots[i]);
      }
    used_before += all;
    base += kPlan * places;
    if (min(base, n_pages) - used_before >= enough) break;   // uniform over the CTA
  }
  return used_before;
}

__device__ __forceinline__ void record(int32_t* status, int32_t bits) {
  if (status) atomicOr(status, bits);
}

// refs and lens of `in` to `out`, by the CTAs behind the planning one.
__device__ __forceinline__ void copy_state(const tq_pages& in, const tq_pages& out, bool refs) {
  if (in.table == out.table) return;
  const int64_t at = static_cast<int64_t>(blockIdx.x - 1) * blockDim.x + threadIdx.x;
  const int64_t step = static_cast<int64_t>(gridDim.x - 1) * blockDim.x;
  for (int64_t i = at; i < in.n_seqs; i += step) out.lens[i] = in.lens[i];
  if (refs)
    for (int64_t i = at; i < in.n_pages; i += step) out.refs[i] = in.refs[i];
}

// The rows of sequences list[0..n) (no list: of all), by the CTAs behind the
// planning one, a warp per row: every entry that the length covers is a page
// that somebody owns.
__device__ __forceinline__ void check_rows(const tq_pages& in, const int32_t* list, int64_t n, const Ws& w) {
  constexpr int kEach = 8;                     // entries of a lane in flight
  const int others = gridDim.x - 1, lane = threadIdx.x % 32;
  int bad = 0;
  for (int64_t i = static_cast<int64_t>(threadIdx.x / 32) * others + blockIdx.x - 1; i < n; i += 32 * others) {
    const int64_t s = list ? list[i] : i;
    if (s < 0 || s >= in.n_seqs) continue;     // the plan's own check
    const int64_t len = in.lens[s];
    const int64_t pages = len <= 0 ? 0 : min((len + in.page_size - 1) / in.page_size, in.max_pages);
    const int32_t* row = in.table + s * in.max_pages;
    for (int64_t j0 = lane; j0 < pages; j0 += 32 * kEach) {
      int32_t page[kEach];
#pragma unroll
      for (int k = 0; k < kEach; ++k) page[k] = j0 + 32 * k < pages ? row[j0 + 32 * k] : row[j0];
#pragma unroll
      for (int k = 0; k < kEach; ++k) bad |= page[k] < 0 || page[k] >= in.n_pages || in.refs[page[k]] <= 0;
    }
  }
  bad = __syncthreads_or(bad);
  if (threadIdx.x == 0) {
    w.head[8 + blockIdx.x - 1] = bad;
    if (bad) record(in.status, kStatusPages);
  }
}
// Whether one of `checkers` CTAs met a bad row; called by a whole CTA.
__device__ __forceinline__ bool rows_bad(const Ws& w, int checkers) {
  int bad = 0;
  for (int i = threadIdx.x; i < checkers; i += kRowThreads) bad |= w.head[8 + i];
  return __syncthreads_or(bad) != 0;
}
// No moves, where a call is not done after all.
__device__ __forceinline__ void no_moves(int32_t* moves, int64_t n) {
  for (int64_t k = static_cast<int64_t>(blockIdx.x) * kRowThreads + threadIdx.x; k < 2 * n;
       k += static_cast<int64_t>(gridDim.x) * kRowThreads)
    moves[k] = -1;
}

__device__ __forceinline__ void clear_map(const Ws& w, int64_t n_seqs) {
  for (int64_t i = threadIdx.x; i < n_seqs; i += kPlan) w.map[i] = -1;
  if (threadIdx.x == 0) w.head[0] = w.head[1] = w.head[2] = 0;
}

__global__ void __launch_bounds__(kPlan) k_plan_fork(tq_pages in, tq_pages out, int n, const int32_t* src,
                                                     const int32_t* dst, int32_t* moves, void* ws) {
  wait_for_stream();
  const Ws w = ws_of(ws, in.n_seqs, n);
  if (blockIdx.x > 0) {
    copy_state(in, out, true);
    return check_rows(in, src, n, w);
  }
  __shared__ int sums[32];
  clear_map(w, in.n_seqs);
  __syncthreads();
  const int64_t cap = in.max_pages * in.page_size;
  int bad = 0, total = 0;
  for (int i0 = 0; i0 < n; i0 += kPlan) {
    const int i = i0 + threadIdx.x;
    int part = 0;
    if (i < n) {
      const int64_t s = src[i], d = dst[i];
      if (s < 0 || s >= in.n_seqs || d < 0 || d >= in.n_seqs || in.lens[d] != 0) {
        bad = 1;
      } else {
        const int len = in.lens[s];
        bad |= len < 0 || len > cap || atomicExch(w.map + d, i) != -1;
        w.len[i] = len;
        part = len > 0 && len % in.page_size != 0;
      }
    }
    int all;
    const int rank = cta_scan(part, sums, &all);
    if (i < n) w.off[i] = part ? total + rank : -1;
    total += all;
  }
  const int n_pages = static_cast<int>(in.n_pages);        // at most 2^30
  int found = 0;
  if (total > 0) {
    over_pages(in.refs, n_pages, total, sums, [&](int page, bool used, int, int rank) {
      if (!used && rank < total) {
        w.list[rank] = page;
        ++found;
      }
    });
  }
  const int any_bad = __syncthreads_or(bad);
  int got;
  cta_scan(found, sums, &got);
  const bool fail = any_bad || got < total;
  if (threadIdx.x == 0) {
    w.head[0] = fail;
    if (any_bad) record(in.status, kStatusIndex);
    else if (fail) record(in.status, kStatusNoPages);
  }
  for (int k = (fail ? 0 : total) + static_cast<int>(threadIdx.x); k < n; k += kPlan) moves[2 * k] = moves[2 * k + 1] = -1;
  if (fail) return;
  for (int i = threadIdx.x; i < n; i += kPlan) {
    const int rank = w.off[i];
    if (rank < 0) continue;
    moves[2 * rank] = in.table[src[i] * in.max_pages + w.len[i] / in.page_size];
    moves[2 * rank + 1] = w.list[rank];
  }
}

__global__ void __launch_bounds__(kRowThreads) k_apply_fork(tq_pages in, tq_pages out, int n, const int32_t* src,
                                                            int32_t* moves, int checkers, bool same, void* ws) {
  wait_for_stream();
  const Ws w = ws_of(ws, in.n_seqs, n);
  const bool bad = rows_bad(w, checkers), fail = bad || w.head[0] != 0;
  if (bad) no_moves(moves, n);
  for (int64_t s = blockIdx.x; s < in.n_seqs; s += gridDim.x) {
    const int i = fail ? -1 : w.map[s];
    int32_t* to = out.table + s * in.max_pages;
    if (i < 0) {
      if (!same)
        for (int64_t j = threadIdx.x; j < in.max_pages; j += kRowThreads) to[j] = in.table[s * in.max_pages + j];
      continue;
    }
    const int32_t* from = in.table + src[i] * in.max_pages;
    const int len = w.len[i], full = len / in.page_size, rank = w.off[i];
    for (int64_t j = threadIdx.x; j < in.max_pages; j += kRowThreads) {
      int32_t page = -1;
      if (j < full) {
        page = from[j];
        atomicAdd(out.refs + page, 1);
      } else if (j == full && rank >= 0) {
        page = w.list[rank];
        out.refs[page] = 1;
      }
      to[j] = page;
    }
    if (threadIdx.x == 0) out.lens[s] = len;
  }
}

__global__ void __launch_bounds__(kPlan) k_plan_extend(tq_pages in, tq_pages out, int n, const int32_t* seqs,
                                                       const int32_t* more, int64_t n_slots, void* ws) {
  wait_for_stream();
  if (blockIdx.x > 0) return copy_state(in, out, true);
  __shared__ int sums[32];
  __shared__ long long lsums[32];
  const Ws w = ws_of(ws, in.n_seqs, n);
  clear_map(w, in.n_seqs);
  __syncthreads();
  const int64_t cap = min(in.max_pages * in.page_size, static_cast<int64_t>(0x7fffffff));
  int bad = 0;
  long long total = 0, tokens = 0;
  for (int i0 = 0; i0 < n; i0 += kPlan) {
    const int i = i0 + threadIdx.x;
    long long need = 0, t = 0;
    if (i < n) {
      const int64_t s = seqs[i];
      t = more[i];
      if (s < 0 || s >= in.n_seqs || t < 0) {
        bad = 1;
        t = 0;
      } else {
        const int64_t len = in.lens[s];
        if (len < 0 || len + t > cap || atomicExch(w.map + s, i) != -1) {
          bad = 1;
          t = 0;
        } else {
          const int64_t have = (len + in.page_size - 1) / in.page_size;
          need = (len + t + in.page_size - 1) / in.page_size - have;
          if (t > 0 && len % in.page_size) {   // the tail goes on in a page that must be this sequence's alone
            const int64_t page = in.table[s * in.max_pages + have - 1];
            bad |= page < 0 || page >= in.n_pages || in.refs[page] != 1;
          }
          w.len[i] = static_cast<int32_t>(len);
        }
      }
    }
    long long all, all_t;
    const long long off = cta_scan(need, lsums, &all);
    const long long at = cta_scan(t, lsums, &all_t);
    if (i < n) {
      w.off[i] = static_cast<int32_t>(min(total + off, static_cast<long long>(0x7fffffff)));
      w.tok[i] = static_cast<int32_t>(min(tokens + at, static_cast<long long>(0x7fffffff)));
    }
    total += all;
    tokens += all_t;
  }
  if (n_slots >= 0 && tokens > n_slots) bad = 1;
  const int n_pages = static_cast<int>(in.n_pages);        // at most 2^30
  int found = 0;
  if (total > 0 && total <= n_pages) {
    over_pages(in.refs, n_pages, static_cast<int>(total), sums, [&](int page, bool used, int, int rank) {
      if (!used && rank < total) {
        w.list[rank] = page;
        ++found;
      }
    });
  }
  const int any_bad = __syncthreads_or(bad);
  int got;
  cta_scan(found, sums, &got);
  if (threadIdx.x == 0) {
    const bool fail = any_bad || got < total;
    w.head[0] = fail;
    w.head[2] = fail ? 0 : static_cast<int32_t>(min(tokens, static_cast<long long>(0x7fffffff)));
    if (any_bad) record(in.status, kStatusIndex);
    else if (fail) record(in.status, kStatusNoPages);
  }
}

__global__ void __launch_bounds__(kRowThreads) k_apply_extend(tq_pages in, tq_pages out, int n, const int32_t* more,
                                                              int64_t* slots, int64_t n_slots, bool same, void* ws) {
  wait_for_stream();
  const Ws w = ws_of(ws, in.n_seqs, n);
  const bool fail = w.head[0] != 0;
  if (slots)
    for (int64_t k = w.head[2] + static_cast<int64_t>(blockIdx.x) * kRowThreads + threadIdx.x; k < n_slots;
         k += static_cast<int64_t>(gridDim.x) * kRowThreads)
      slots[k] = -1;
  for (int64_t s = blockIdx.x; s < in.n_seqs; s += gridDim.x) {
    const int i = fail ? -1 : w.map[s];
    const int32_t* from = in.table + s * in.max_pages;
    int32_t* to = out.table + s * in.max_pages;
    if (!same)
      for (int64_t j = threadIdx.x; j < in.max_pages; j += kRowThreads) to[j] = from[j];
    if (i < 0) continue;
    const int64_t len = w.len[i], t = more[i], ps = in.page_size;
    const int64_t have = (len + ps - 1) / ps, need = (len + t + ps - 1) / ps - have;
    const int32_t* list = w.list + w.off[i];
    __syncthreads();                           // the row's copy stands before its new entries
    for (int64_t j = threadIdx.x; j < need; j += kRowThreads) {
      to[have + j] = list[j];
      out.refs[list[j]] = 1;
    }
    if (slots)
      for (int64_t k = threadIdx.x; k < t; k += kRowThreads) {
        const int64_t pos = len + k, at = pos / ps;
        const int64_t page = at < have ? from[at] : list[at - have];
        slots[w.tok[i] + k] = page * ps + pos % ps;
      }
    if (threadIdx.x == 0) out.lens[s] = static_cast<int32_t>(len + t);
  }
}

__global__ void __launch_bounds__(kPlan) k_plan_free(tq_pages in, tq_pages out, int n, const int32_t* seqs, void* ws) {
  wait_for_stream();
  const Ws w = ws_of(ws, in.n_seqs, n);
  if (blockIdx.x > 0) {
    copy_state(in, out, true);
    return check_rows(in, seqs, n, w);
  }
  clear_map(w, in.n_seqs);
  __syncthreads();
  int bad = 0;
  for (int i = threadIdx.x; i < n; i += kPlan) {
    const int64_t s = seqs[i];
    if (s < 0 || s >= in.n_seqs) bad = 1;
    else w.map[s] = 1;                         // named twice: the same mark
  }
  bad = __syncthreads_or(bad);
  if (threadIdx.x == 0) {
    w.head[0] = bad;
    if (bad) record(in.status, kStatusIndex);
  }
}

__global__ void __launch_bounds__(kRowThreads) k_apply_free(tq_pages in, tq_pages out, int n, int checkers,
                                                            bool same, void* ws) {
  wait_for_stream();
  const Ws w = ws_of(ws, in.n_seqs, n);
  const bool fail = rows_bad(w, checkers) || w.head[0] != 0;
  for (int64_t s = blockIdx.x; s < in.n_seqs; s += gridDim.x) {
    const bool ends = !fail && w.map[s] == 1;
    const int32_t* from = in.table + s * in.max_pages;
    int32_t* to = out.table + s * in.max_pages;
    const int64_t len = in.lens[s];
    const int64_t pages = len <= 0 ? 0 : min((len + in.page_size - 1) / in.page_size, in.max_pages);
    __syncthreads();                           // every thread has the length before it is cleared
    if (!ends && same) continue;
    for (int64_t j = threadIdx.x; j < in.max_pages; j += kRowThreads) {
      const int32_t page = from[j];
      if (ends && j < pages) atomicSub(out.refs + page, 1);
      to[j] = ends ? -1 : page;
    }
    if (ends && threadIdx.x == 0) out.lens[s] = 0;
  }
}

__global__ void __launch_bounds__(kPlan) k_plan_compact(tq_pages in, tq_pages out, int32_t* moves, int64_t most,
                                                        void* ws) {
  wait_for_stream();
  const Ws w = ws_of(ws, in.n_seqs, 0);
  if (blockIdx.x > 0) {
    copy_state(in, out, false);
    return check_rows(in, nullptr, in.n_seqs, w);
  }
  __shared__ int sums[32];
  const int n_pages = static_cast<int>(in.n_pages), all = n_pages + 1;     // at most 2^30
  const int used = over_pages(in.refs, n_pages, all, sums, [](int, bool, int, int) {});
  // the k-th free place before `used` and the k-th used page from there on
  int holes = 0, count;
  over_pages(in.refs, n_pages, all, sums, [&](int page, bool u, int, int free_rank) {
    if (page < used && !u) {
      moves[2 * static_cast<int64_t>(free_rank) + 1] = page;
      ++holes;
    }
    if (page >= used) w.list[page] = -1;
  });
  cta_scan(holes, sums, &count);
  over_pages(in.refs, n_pages, all, sums, [&](int page, bool u, int used_rank, int) {
    // count used pages stand behind; used - count before
    if (page >= used && u) moves[2 * static_cast<int64_t>(used_rank - (used - count))] = page;
  });
  __syncthreads();
  for (int64_t k = threadIdx.x; k < most; k += kPlan) {
    if (k < count) w.list[moves[2 * k]] = moves[2 * k + 1];
    else moves[2 * k] = moves[2 * k + 1] = -1;
  }
  if (threadIdx.x == 0) {
    w.head[0] = count;
    w.head[1] = used;
  }
}

__global__ void __launch_bounds__(kRowThreads) k_apply_compact(tq_pages in, tq_pages out, int32_t* moves, int64_t most,
                                                               int checkers, bool same, void* ws) {
  wait_for_stream();
  const Ws w = ws_of(ws, in.n_seqs, 0);
  const bool bad = rows_bad(w, checkers);
  const int64_t count = w.head[0], used = w.head[1];
  const int64_t at = static_cast<int64_t>(blockIdx.x) * kRowThreads + threadIdx.x;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kRowThreads;
  if (bad) {                                   // out takes in's contents
    no_moves(moves, most);
    if (same) return;
    for (int64_t p = at; p < in.n_pages; p += step) out.refs[p] = in.refs[p];
    for (int64_t s = blockIdx.x; s < in.n_seqs; s += gridDim.x)
      for (int64_t j = threadIdx.x; j < in.max_pages; j += kRowThreads)
        out.table[s * in.max_pages + j] = in.table[s * in.max_pages + j];
    return;
  }
  // a pair's two counts belong to one thread, so working in place is safe
  for (int64_t k = at; k < count; k += step) {
    const int32_t high = moves[2 * k], hole = moves[2 * k + 1];
    const int32_t v = in.refs[high];
    out.refs[hole] = v;
    out.refs[high] = 0;
  }
  if (!same)
    for (int64_t p = at; p < in.n_pages; p += step) {
      const int32_t v = in.refs[p];
      if ((p < used) == (v > 0)) out.refs[p] = v;
    }
  for (int64_t s = blockIdx.x; s < in.n_seqs; s += gridDim.x) {
    const int64_t len = in.lens[s];
    const int64_t pages = len <= 0 ? 0 : min((len + in.page_size - 1) / in.page_size, in.max_pages);
    for (int64_t j = threadIdx.x; j < in.max_pages; j += kRowThreads) {
      int32_t page = -1;
      if (j < pages) {
        page = in.table[s * in.max_pages + j];
        if (page >= used) page = w.list[page];
      }
      out.table[s * in.max_pages + j] = page;
    }
  }
}

// Pages by moves.  Every CTA packs 1024 moves at a time into the list of those
// that are wanted, and takes every gridDim-th chunk of their bytes, so a list
// that is mostly -1 costs its reading only.
constexpr int kCopyThreads = 256, kGroup = 1024, kUnroll = 4;

template <typename W>
__global__ void __launch_bounds__(kCopyThreads) k_copy_pages(uint8_t* base, int64_t n_layers, int64_t layer_stride,
                                                             int64_t page_bytes, int64_t n_pages,
                                                             const int32_t* moves, int64_t n_moves) {
  wait_for_stream();
  __shared__ int2 list[kGroup];
  __shared__ int sums[kCopyThreads / 32];
  constexpr int64_t kChunk = static_cast<int64_t>(kCopyThreads) * kUnroll * sizeof(W);
  const int64_t chunks = (page_bytes + kChunk - 1) / kChunk, per_move = chunks * n_layers;
  int64_t skip = blockIdx.x;                   // this CTA's next unit, counted from the group's first
  for (int64_t m0 = 0; m0 < n_moves; m0 += kGroup) {
    int2 mv[kGroup / kCopyThreads];
    int good = 0;
#pragma unroll
    for (int i = 0; i < kGroup / kCopyThreads; ++i) {
      const int64_t m = m0 + threadIdx.x * (kGroup / kCopyThreads) + i;
      mv[i] = m < n_moves ? make_int2(moves[2 * m], moves[2 * m + 1]) : make_int2(-1, -1);
      if (mv[i].x < 0 || mv[i].x >= n_pages || mv[i].y < 0 || mv[i].y >= n_pages || mv[i].x == mv[i].y) mv[i].x = -1;
      good += mv[i].x >= 0;
    }
    int total;
    int at = cta_scan(good, sums, &total);     // its first barrier: the list of the group before is done with
#pragma unroll
    for (int i = 0; i < kGroup / kCopyThreads; ++i)
      if (mv[i].x >= 0) list[at++] = mv[i];
    __syncthreads();
    const int64_t units = total * per_move;
    for (; skip < units; skip += gridDim.x) {
      const int64_t k = skip / per_move, rest = skip - k * per_move, layer = rest / chunks, ch = rest - layer * chunks;
      uint8_t* l = base + layer * layer_stride;
      const W* from = reinterpret_cast<const W*>(l + list[k].x * page_bytes + ch * kChunk);
      W* to = reinterpret_cast<W*>(l + list[k].y * page_bytes + ch * kChunk);
      const int64_t words = min(kChunk, page_bytes - ch * kChunk) / static_cast<int64_t>(sizeof(W));
      W v[kUnroll];
#pragma unroll
      for (int i = 0; i < kUnroll; ++i)
        if (threadIdx.x + i * kCopyThreads < words) v[i] = __ldcs(from + threadIdx.x + i * kCopyThreads);
#pragma unroll
      for (int i = 0; i < kUnroll; ++i)
        if (threadIdx.x + i * kCopyThreads < words) to[threadIdx.x + i * kCopyThreads] = v[i];
    }
    skip -= units;
  }
}

dim3 rows_grid(const tq_pages& p) { return dim3(static_cast<unsigned>(std::min<int64_t>(p.n_seqs, 148 * 16))); }
// the planning CTA, and the ones that check `rows` rows, and copy where in and out differ
dim3 plan_grid(const tq_pages& p, bool same, int64_t rows) {
  const int64_t copies = same ? 0 : (p.n_seqs + p.n_pages + kPlan - 1) / kPlan;
  return dim3(1 + static_cast<unsigned>(std::min<int64_t>(kOthers, std::max(rows, copies))));
}
bool is_same(const tq_pages& a, const tq_pages& b) { return a.table == b.table; }

}  // namespace

size_t pages_ws_bytes(const tq_pages& p, int64_t n) {
  return round16(static_cast<size_t>(kHead + p.n_seqs + 3 * n + p.n_pages) * 4);
}

int launch_pages_extend(const tq_pages& in, const tq_pages& out, int64_t n, const int32_t* seqs,
                        const int32_t* new_tokens, int64_t* slots, int64_t n_slots, void* ws, void* stream) {
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool same = is_same(in, out);
  const int k = static_cast<int>(n);
  if (int e = launch_dependent(k_plan_extend, plan_grid(in, same, 0), dim3(kPlan), 0, st, in, out, k, seqs, new_tokens,
                               slots ? n_slots : -1, ws))
    return e;
  return launch_dependent(k_apply_extend, rows_grid(in), dim3(kRowThreads), 0, st, in, out, k, new_tokens, slots,
                          n_slots, same, ws);
}

int launch_pages_fork(const tq_pages& in, const tq_pages& out, int64_t n, const int32_t* src, const int32_t* dst,
                      int32_t* moves, void* ws, void* stream) {
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool same = is_same(in, out);
  const int k = static_cast<int>(n);
  const dim3 plan = plan_grid(in, same, n);
  if (int e = launch_dependent(k_plan_fork, plan, dim3(kPlan), 0, st, in, out, k, src, dst, moves, ws)) return e;
  return launch_dependent(k_apply_fork, rows_grid(in), dim3(kRowThreads), 0, st, in, out, k, src, moves,
                          static_cast<int>(plan.x - 1), same, ws);
}

int launch_pages_free(const tq_pages& in, const tq_pages& out, int64_t n, const int32_t* seqs, void* ws,
                      void* stream) {
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool same = is_same(in, out);
  const int k = static_cast<int>(n);
  const dim3 plan = plan_grid(in, same, n);
  if (int e = launch_dependent(k_plan_free, plan, dim3(kPlan), 0, st, in, out, k, seqs, ws)) return e;
  return launch_dependent(k_apply_free, rows_grid(in), dim3(kRowThreads), 0, st, in, out, k,
                          static_cast<int>(plan.x - 1), same, ws);
}

int launch_pages_compact(const tq_pages& in, const tq_pages& out, int32_t* moves, void* ws, void* stream) {
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool same = is_same(in, out);
  const dim3 plan = plan_grid(in, same, in.n_seqs);
  const int64_t most = std::max<int64_t>(1, in.n_pages / 2);
  if (int e = launch_dependent(k_plan_compact, plan, dim3(kPlan), 0, st, in, out, moves, most, ws)) return e;
  return launch_dependent(k_apply_compact, rows_grid(in), dim3(kRowThreads), 0, st, in, out, moves, most,
                          static_cast<int>(plan.x - 1), same, ws);
}

int launch_pages_copy(void* base, int64_t n_layers, int64_t layer_stride, int64_t page_bytes, int64_t n_pages,
                      const int32_t* moves, int64_t n_moves, void* stream) {
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool wide = (reinterpret_cast<uintptr_t>(base) | static_cast<uintptr_t>(layer_stride) |
                     static_cast<uintptr_t>(page_bytes)) % 16 == 0;
  const int64_t chunk = kCopyThreads * kUnroll * (wide ? 16 : 4);
  const int64_t most = 148 * 8;                // CTAs; the moves are cut to as many, so that the product fits
  const int64_t units = std::min(n_moves, most) * n_layers * ((page_bytes + chunk - 1) / chunk);
  const dim3 grid(static_cast<unsigned>(std::min(units, most)));
  return launch_dependent(wide ? k_copy_pages<uint4> : k_copy_pages<uint32_t>, grid, dim3(kCopyThreads), 0, st,
                          static_cast<uint8_t*>(base), n_layers, layer_stride, page_bytes, n_pages, moves, n_moves);
}

}  // namespace tq
