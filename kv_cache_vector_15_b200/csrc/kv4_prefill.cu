// Attention of many query rows over the paged 4-bit cache: chunks of a prompt
// behind a cached prefix, or many decoder tokens against an encoder's states
// (bf16 rows; decode-sized calls and fp32 rows go to the other kernel).
//
// Here the work is products: 4 d per query row and key against 9 d / 8 bytes
// per key that 256 rows share, so the tensor cores set the floor.  One CTA per
// SM works on 256 query rows (two tiles of 128; the q heads of a kv head are
// rows of the same tile) and runs through the keys in tiles of 128:
//
//   8 warps unpack   codes and pairs -> binary16 operands, 128-byte swizzled (a
//                    thread takes 64 coordinates of a token)
//   1 warp issues    S = Q K^T (tcgen05, operands in shared memory) and
//                    O += P V (P from tensor memory, V as it was unpacked:
//                    keys down, coordinates across, an MN-major operand)
//   2 x 4 warps      softmax, a thread per row: maximum, weights, sum; P goes
//                    to tensor memory over S's columns
//
// so while one tile's softmax runs, the other's products do.
//
// Precision.  vhat = z + s c and p enter in binary16: its 11 bits keep the
// result's error well below a bf16 output's rounding, where bf16 operands
// would double it.  For the logits that is not enough (rounding khat to 11 bits
// moved the log-sum-exp by 1.3e-5 of its size): s (c - 8) is taken as two
// binary16 numbers, the rounded product and its exact remainder, and z + 8 s,
// times the sum of q over the group, as 16 more terms of the sum (three of
// products of high and low parts per group), so the logits have 22 bits.  q,
// scaled per row by a power of two, loses nothing of its 8 bits.  The second
// pass over K costs tensor time, which the softmax's issue slots and
// exponentials hide.  p is 2^(logit - m + 7), m a running maximum that is
// renewed when a logit passes it by 2^8: p stays below 2^15, and what is 2^-31
// of the maximum still counts (weights spread over 10^5 tokens beside a
// dominant one).  Rescaling O in tensor memory is the rare case then.
//
// d = 256 has 128 rows and 64 keys per tile: O and S fill the tensor memory's
// columns, Q, K and two stages of V the shared memory.
//
// Split: the line of key tiles of all (sequence, kv head, 256 rows) units is
// cut into equal parts, one per CTA, and partial sums are joined by a second
// kernel, as in the decode kernel; units alone would leave SMs idle in the
// last wave.
//
// Measured, bf16, 4 sequences of 171 to 512 new tokens behind 4099 to 8200, 8 kv
// heads of 4 query heads, d = 128 (122 GFLOP): 0.207 to 0.225 ms = 540 to 590 TFLOP/s,
// 34 to 37 % of the GEMM rate; the tensor pipe is active in 50 % of the cycles.  A tile of
// 256 rows and 128 keys takes 6500 clocks: 4000 of products
// (two passes over K; operands in shared memory at N = 128 use all of its
// bandwidth), the rest waiting for K to be unpacked, weights and query rows.
// Waiting for K before the first Q tile's values instead of behind them: 0.238 ms;
// unpacking K's low parts under the last products' high ones 0.23 (their stores
// take shared-memory bandwidth from the products).  A product of 128 x 128 x 16 takes about 80 clocks; with 64
// keys a tile and Q in tensor memory one of 128 x 64 x 16 took about as long
// (0.29 ms), so tiles stay 128 keys wide.  The query rows on the few-row kernel's
// tiles: 2.1 ms; khat rounded once 0.34 at the time, with four unpacking warps.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "kv4_internal.h"
#include "kv4_line.cuh"
#include "sm100.cuh"
#include "tq_internal.h"

namespace tq {
namespace {

using namespace sm100;

constexpr int kCtas = 148;
// What a unit costs besides its tiles, in tiles.  With 1, 3 and 6: the case above 223, 218, 217 us, 16 sequences of 64
// rows behind 1000 tokens 61.0, 58.4, 57.8, 64 of 10 .. 32 rows behind 130 .. 2000 152, 119, 126, one of 400 30.9, 31.0, 33.9.
constexpr int kCost = 3;
constexpr float kShift = 7.f;                  // p = 2^(logit - m + kShift)

__host__ __device__ constexpr int q_tiles_of(int d) { return d == 256 ? 1 : 2; }
__host__ __device__ constexpr int keys_of(int d) { return d == 256 ? 64 : 128; }

// MN-major operand, 128-byte swizzle: rows (keys) 128 B apart, 8-key groups
// 1024 B apart, chunks of 64 coordinates `lbo` bytes apart.
__device__ __forceinline__ uint64_t desc_mn_sw128(uint32_t saddr, uint32_t lbo) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr >> 4) & 0x3FFFu);
  d |= static_cast<uint64_t>((lbo >> 4) & 0x3FFFu) << 16;
  d |= static_cast<uint64_t>((1024u >> 4) & 0x3FFFu) << 32;
  d |= static_cast<uint64_t>(1u) << 46;
  d |= static_cast<uint64_t>(2u) << 61;
  return d;
}

// K-major operand of 16 terms, not swizzled: 8 rows x 16 bytes contiguous, the
// second 8 terms 128 B behind the first, 8-row groups 256 B apart.
__device__ __forceinline__ uint64_t desc_plain16(uint32_t saddr) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr >> 4) & 0x3FFFu);
  d |= static_cast<uint64_t>(128u >> 4) << 16;
  d |= static_cast<uint64_t>(256u >> 4) << 32;
  d |= static_cast<uint64_t>(1u) << 46;
  return d;
}

// Products and commits by the lane whose `leader` is set, in code that the whole
// warp runs: descriptors stay in uniform registers (a branch for one lane costs
// a move per operand, about 100 cycles per product here).
__device__ __forceinline__ void mma_ss(uint32_t leader, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc),
      "r"(leader)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t leader, uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(acc),
      "r"(leader)
      : "memory");
}
__device__ __forceinline__ void commit(uint32_t leader, uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar)), "r"(leader)
      : "memory");
}
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r;
}

__device__ __forceinline__ uint32_t h2_add(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("add.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t h2_fma(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}
__device__ __forceinline__ uint32_t h2_mul(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t h2_min(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("min.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// The 8 codes of a word as binary16 c - kBias, in the order 0 4 1 5 2 6 3 7 (in
// which Q and O stand too): 0x6400 | c is 1024 + c, 0x6400 | 16 c is 1024 + 16 c.
template <int kBias>
__device__ __forceinline__ void codes8(uint32_t w, uint32_t (&c)[4]) {
  constexpr uint32_t kMinus = kBias == 0 ? 0xe400e400u : 0xe408e408u;        // - 1024, - 1032
  constexpr uint32_t kMinus16 = kBias == 0 ? 0xd400d400u : 0xd480d480u;      // - 64, - 72
  const uint32_t v = w >> 8;
  c[0] = h2_add((w & 0x000f000fu) | 0x64006400u, kMinus);
  c[1] = h2_fma((w & 0x00f000f0u) | 0x64006400u, 0x2c002c00u, kMinus16);     // / 16
  c[2] = h2_add((v & 0x000f000fu) | 0x64006400u, kMinus);
  c[3] = h2_fma((v & 0x00f000f0u) | 0x64006400u, 0x2c002c00u, kMinus16);
}
__device__ __forceinline__ uint32_t high_low(float x) {      // binary16 high part and what it leaves
  const float h = __half2float(__float2half_rn(x));
  return pack_f16(h, x - h);
}

template <int D>
struct Shape {
  static constexpr int QT = q_tiles_of(D), KT = keys_of(D), CH = D / 64;
  static constexpr int kQ = CH * 128 * 128;              // bytes of a Q tile
  static constexpr int kKV = CH * KT * 128;              // bytes of K's high or low parts, or of a stage of V
  static constexpr int kQx = 128 * 32, kKx = KT * 32;    // the 16 more terms
  static constexpr int kAtQx = QT * kQ + 4 * kKV;        // behind Q, K high, K low, V, V
  static constexpr int kBars = kAtQx + QT * kQx + kKx;   // barriers behind the operands
  static constexpr int kLost = CH * KT / 32;             // words of a stage's marks of NaN values: a bit per group and token
  static constexpr int kBytes = kBars + 256 + 1024;      // and slack for the 1024-byte alignment
  static_assert(144 + 2 * kLost * 4 <= 256, "the marks fit behind the barriers");
  static constexpr int kSmem = kBytes < 120 * 1024 ? 120 * 1024 : kBytes;   // one CTA per SM: it takes all of TMEM
  static constexpr int kSoft = 4 * QT;                   // softmax warps
  static constexpr int kUnpack = KT * CH / 32;           // unpacking warps: a thread per token and 64 coordinates
  static constexpr int kThreads = (kSoft + kUnpack + 1) * 32;
  static constexpr int kO = QT * KT;                     // first TMEM column of O; S tiles stand before
};

template <int D>
__global__ void __launch_bounds__(Shape<D>::kThreads, 1) k_kv4_prefill(const __grid_constant__ Params P) {
  using Z = Shape<D>;
  constexpr int QT = Z::QT, KT = Z::KT, R = 128 * QT;
  extern __shared__ uint8_t raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* sq = sm;
  uint8_t* sk = sm + QT * Z::kQ;
  uint8_t* sv = sk + 2 * Z::kKV;
  uint8_t* sqx = sm + Z::kAtQx;
  uint8_t* skx = sqx + QT * Z::kQx;
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + Z::kBars);
  uint64_t *q_full = bars, *s_full = bars + 2, *p_full = bars + 4, *o_done = bars + 6, *k_full = bars + 8,
           *k_free = bars + 10, *v_full = bars + 12, *v_free = bars + 14, *drain = bars + 16;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 17);
  uint32_t* lost = reinterpret_cast<uint32_t*>(bars + 18);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int worker = blockIdx.x;

  // of the 16 more terms, 3 per group are written later; the others stay zero
  for (int i = threadIdx.x; i < (QT * Z::kQx + Z::kKx) / 16; i += Z::kThreads)
    reinterpret_cast<uint4*>(sqx)[i] = make_uint4(0, 0, 0, 0);
  fence_proxy_async_smem();
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(q_full + i, 128);
      mbar_init(s_full + i, 1);
      mbar_init(p_full + i, 128);
      mbar_init(o_done + i, 1);
      mbar_init(k_full + i, Z::kUnpack * 32);
      mbar_init(k_free + i, 1);
      mbar_init(v_full + i, Z::kUnpack * 32);
      mbar_init(v_free + i, 1);
    }
    mbar_init(drain, 1);
    mbar_fence_init();
  }
  // Tensor memory is taken behind the wait: a kernel before this one that has let its dependents start may itself still
  // want some, and would get none from a CTA that holds all of it and waits for that kernel's end.
  wait_for_stream();
  if (warp == Z::kSoft + Z::kUnpack) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  const Part part = part_of<KT, kCost>(P, worker, R, 1);
  int32_t* desc = P.desc + worker * kDescInts;
  if (threadIdx.x == 0) desc[0] = 0;
  bool ok = true;
  Piece u = piece_at(part);
  uint32_t tiles_done = 0;                     // key tiles of this CTA so far (units without tiles have none)
  uint32_t units_done[2] = {0, 0};             // units in which Q tile 0, 1 took part ...
  uint32_t q_tiles_done[2] = {0, 0};           // ... and their key tiles

  // where term i of a row's 16 more terms stands
  auto at_more = [](int row, int i) { return (row / 8) * 256 + (row % 8) * 16 + (i / 8) * 128 + (i % 8) * 2; };
  // a wait that a whole warp makes: all of its lanes go on, or none
  auto wait_warp = [&](uint64_t* bar, uint32_t parity) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity & 1u, P.limit)) != 0;
  };
  Seq q = {};                                  // of the piece at hand
  int h = 0, rt = 0, t0 = 0, n_tiles = 0, n_rows = 0, nqt = 0;
  bool whole = false;
  // Every role runs through the same pieces.
  auto units = [&](auto role) {
    bool more = part.a < part.b && settle<KT, kCost>(P, R, part.b, u);
    while (more && ok) {
      q = u.q;
      h = u.h;
      rt = u.rt;
      t0 = u.t0;
      n_tiles = u.n_tiles;
      n_rows = q.n * P.g;
      nqt = QT == 1 || n_rows - rt * R <= 128 ? 1 : 2;
      whole = u.whole;
      role();
      if (!whole && u.first && threadIdx.x == 0) describe(desc, u, part.share, worker);
      tiles_done += n_tiles;
      if (n_tiles > 0)
        for (int qt = 0; qt < nqt; ++qt) {
          ++units_done[qt];
          q_tiles_done[qt] += n_tiles;
        }
      more = next_piece<KT, kCost>(P, R, part.b, u);
    }
  };

  if (warp < Z::kSoft) {
    units([&]() {
      // ---------------------------------------------------------- softmax --
      const int qt = warp / 4, tid = threadIdx.x - qt * 128;
      if (qt < nqt) {
        const int row = rt * R + qt * 128 + tid;
        const bool live = row < n_rows;
        const int j = live ? row / P.g : q.n - 1, hi_row = live ? row - j * P.g : 0;
        const int64_t orow = static_cast<int64_t>(q.q0 + j) * P.q_heads + h * P.g + hi_row;
        int lo, hi;
        sees(P, q, j, lo, hi);
        float scale = 0.f;
        if (n_tiles > 0) {
          // The warp's 32 rows, D / 8 lanes to a row, scaled by a power of two to below 2^4, in the operand's order; a
          // negative softmax scale changes their sign.
          constexpr int kLanes = D / 8, kRows = 32 / kLanes, kBatch = 8;
          const int l8 = lane % kLanes, rsub = lane / kLanes, g = l8 / 8;
          uint8_t* dst = sq + qt * Z::kQ + g * (128 * 128);
          uint8_t* dst_more = sqx + qt * Z::kQx;
#pragma unroll 1
          for (int r0 = 0; r0 < 32; r0 += kRows * kBatch) {
            uint4 w[kBatch];
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
              const int qrow = rt * R + qt * 128 + (warp % 4) * 32 + r0 + k * kRows + rsub;
              const int qj = qrow / P.g;
              w[k] = make_uint4(0, 0, 0, 0);
              if (qrow < n_rows)
                w[k] = __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(P.q) + (q.q0 + qj) * P.ld_q +
                                                            static_cast<int64_t>(h * P.g + qrow - qj * P.g) * D) + l8);
            }
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
              const int rin = r0 + k * kRows + rsub, tq = (warp % 4) * 32 + rin;       // row in the warp, in the tile
              const uint32_t u[4] = {w[k].x, w[k].y, w[k].z, w[k].w};
              float f[8], top = 0.f;
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                f[2 * e] = __uint_as_float(u[e] << 16);
                f[2 * e + 1] = __uint_as_float(u[e] & 0xffff0000u);
                top = fmaxf(top, fmaxf(fabsf(f[2 * e]), fabsf(f[2 * e + 1])));
              }
#pragma unroll
              for (int o = kLanes / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
              int ex = 0;
              frexpf(top, &ex);
              ex = top > 0.f ? min(4 - ex, 120) : 0;
              const float up = P.scale_log2 < 0.f ? -pow2(ex) : pow2(ex);
#pragma unroll
              for (int e = 0; e < 8; ++e) f[e] *= up;
              *reinterpret_cast<uint4*>(dst + tq * 128 + (((l8 % 8) ^ (tq % 8)) * 16)) =
                  make_uint4(pack_f16(f[0], f[4]), pack_f16(f[1], f[5]), pack_f16(f[2], f[6]), pack_f16(f[3], f[7]));
              float sum = ((f[0] + f[1]) + (f[2] + f[3])) + ((f[4] + f[5]) + (f[6] + f[7]));
#pragma unroll
              for (int o = 4; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
              if (l8 % 8 == 0) {                 // per group: high, high, low part of the sum of q
                const uint32_t hl = high_low(sum);
                *reinterpret_cast<uint16_t*>(dst_more + at_more(tq, 3 * g)) = static_cast<uint16_t>(hl & 0xffffu);
                *reinterpret_cast<uint16_t*>(dst_more + at_more(tq, 3 * g + 1)) = static_cast<uint16_t>(hl & 0xffffu);
                *reinterpret_cast<uint16_t*>(dst_more + at_more(tq, 3 * g + 2)) = static_cast<uint16_t>(hl >> 16);
              }
              // the scale to the thread that has the row
#pragma unroll
              for (int x = 0; x < kRows; ++x) {
                const float sc = fabsf(P.scale_log2) * pow2(-__shfl_sync(0xffffffffu, ex, x * kLanes));
                if (lane == r0 + k * kRows + x) scale = sc;
              }
            }
          }
          fence_proxy_async_smem();
          mbar_arrive(q_full + qt);
        }
        const uint32_t t_s = tmem + (static_cast<uint32_t>((warp % 4) * 32) << 16) + qt * KT;
        const uint32_t t_o = tmem + (static_cast<uint32_t>((warp % 4) * 32) << 16) + Z::kO + qt * D;
        float m = kLowest, l = 0.f;
        uint32_t lost_groups = 0;              // in which the row sees a NaN value
        for (int i = 0; i < n_tiles; ++i) {
          const uint32_t n = q_tiles_done[qt] + i;
          if (!(ok = wait_warp(s_full + qt, n))) break;
          tc_fence_after();
          const int key0 = (t0 + i) * KT;
          const bool edge = __any_sync(0xffffffffu, key0 < lo || key0 + KT - 1 > hi);
          // the maximum in use, and O with it, after a logit that passes it
          auto renew = [&](float top) {
            const bool grow = top > m + kLazy;
            if (!__any_sync(0xffffffffu, grow)) return true;
            const float f = grow ? ex2(m - top) : 1.f;
            if (grow) m = top;
            l *= f;
            if (i > 0) {
              if (!wait_warp(o_done + qt, n - 1)) return false;
              tc_fence_after();
#pragma unroll 1
              for (int c = 0; c < D; c += 16) {
                uint32_t v[16];
                tmem_ld16(t_o + c, v);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 16; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * f);
                tmem_st16(t_o + c, v);
              }
              tmem_wait_st();
            }
            return true;
          };
          float sum[4] = {0.f, 0.f, 0.f, 0.f};
          if (!edge) {
            float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
            for (int c = 0; c < KT; c += 64) {
              uint32_t v[64];
              tmem_ld32(t_s + c, *reinterpret_cast<uint32_t(*)[32]>(v));
              tmem_ld32(t_s + c + 32, *reinterpret_cast<uint32_t(*)[32]>(v + 32));
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 64; e += 8)
#pragma unroll
                for (int k = 0; k < 4; ++k)
                  top[k] = fmaxf(top[k], fmaxf(__uint_as_float(v[e + 2 * k]), __uint_as_float(v[e + 2 * k + 1])));
            }
            if (!(ok = renew(fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * scale))) break;
            const float off = kShift - m;
#pragma unroll 1
            for (int c = 0; c < KT; c += 32) {             // the weights, over columns that are read already
              uint32_t v[32], w[16];
              tmem_ld32(t_s + c, v);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                const float p0 = ex2(fmaf(__uint_as_float(v[2 * e]), scale, off));
                const float p1 = ex2(fmaf(__uint_as_float(v[2 * e + 1]), scale, off));
                sum[2 * (e & 1)] += p0;
                sum[2 * (e & 1) + 1] += p1;
                w[e] = pack_f16(p0, p1);
              }
              tmem_st16(t_s + c / 2, w);
            }
          } else {                             // the same in two passes, by what the row sees
            float top = -INFINITY;
#pragma unroll 1
            for (int c = 0; c < KT; c += 32) {
              uint32_t v[32];
              tmem_ld32(t_s + c, v);
              tmem_wait_ld();
              const int a = lo - key0 - c, b = hi - key0 - c;
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (e >= a && e <= b) top = fmaxf(top, __uint_as_float(v[e]));
            }
            if (!(ok = renew(top == -INFINITY ? top : top * scale))) break;
            const float off = kShift - m;
#pragma unroll 1
            for (int c = 0; c < KT; c += 32) {
              uint32_t v[32], w[16];
              tmem_ld32(t_s + c, v);
              tmem_wait_ld();
              const int a = lo - key0 - c, b = hi - key0 - c;
#pragma unroll
              for (int e = 0; e < 32; ++e) {
                const float p = e >= a && e <= b ? ex2(fmaf(__uint_as_float(v[e]), scale, off)) : 0.f;
                sum[e & 3] += p;
                v[e] = __float_as_uint(p);
              }
#pragma unroll
              for (int e = 0; e < 16; ++e) w[e] = pack_f16(__uint_as_float(v[2 * e]), __uint_as_float(v[2 * e + 1]));
              tmem_st16(t_s + c / 2, w);
            }
          }
          l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
          tmem_wait_st();
          tc_fence_before();
          // NaN values are zero in V (a weight of zero times NaN would reach the rows that do not see them): the rows that
          // see one look for its mark.  The products wait for V as well, so this wait costs nothing; the marks stand until
          // these weights have been used.
          const uint32_t tile = tiles_done + i;
          if (!(ok = wait_warp(v_full + (tile & 1u), tile >> 1))) break;
          const uint32_t* marks = lost + (tile & 1u) * Z::kLost;
          uint32_t any = 0;
#pragma unroll
          for (int k = 0; k < Z::kLost; ++k) any |= marks[k];
          if (any != 0) {
#pragma unroll 1
            for (int k = 0; k < Z::kLost; ++k) {
              const int first = key0 + k % (KT / 32) * 32, a = max(lo - first, 0), b = min(hi - first, 31);
              if (a <= b && (marks[k] & (0xffffffffu << a) & (0xffffffffu >> (31 - b))) != 0) lost_groups |= 1u << (k / (KT / 32));
            }
          }
          mbar_arrive(p_full + qt);
        }
        if (n_tiles > 0 && ok) {
          ok = wait_warp(o_done + qt, q_tiles_done[qt] + n_tiles - 1);
          tc_fence_after();
        }
        if (ok) {
          const float inv = whole ? (l > 0.f || l != l ? 1.f / l : 0.f) : 1.f;
          // partial sums stand by columns [D + 2][R]: neighbouring threads, neighbouring rows
          float* sums = P.partial + (static_cast<int64_t>(worker) * 2 + (u.first ? 1 : 0)) * R * (D + 4) + qt * 128 + tid;
          __nv_bfloat16* out = static_cast<__nv_bfloat16*>(P.out) + orow * D;
#pragma unroll 1
          for (int c = 0; c < D; c += 32) {
            const float by = (lost_groups >> (c / 64)) & 1u ? __int_as_float(0x7fffffff) : inv;
            uint32_t v[32];
            if (n_tiles > 0) {
              tmem_ld32(t_o + c, v);
              tmem_wait_ld();
            } else {
#pragma unroll
              for (int e = 0; e < 32; ++e) v[e] = 0;
            }
#pragma unroll
            for (int e = 0; e < 32; e += 8) {  // columns 0 1 2 3 ... hold coordinates 0 4 1 5 2 6 3 7 of each 8
              float o[8];
#pragma unroll
              for (int k = 0; k < 8; ++k) o[(k & 1) * 4 + k / 2] = __uint_as_float(v[e + k]) * by;
              if (whole) {
                if (live)
                  *reinterpret_cast<uint4*>(out + c + e) =
                      make_uint4(pack_bf16(o[0], o[1]), pack_bf16(o[2], o[3]), pack_bf16(o[4], o[5]), pack_bf16(o[6], o[7]));
              } else {
#pragma unroll
                for (int k = 0; k < 8; ++k) sums[(c + e + k) * R] = o[k];
              }
            }
          }
          if (!whole) {
            sums[D * R] = m - kShift;          // the sums carry 2^kShift
            sums[(D + 1) * R] = l;
          } else if (live && P.lse) {
            P.lse[orow] = l > 0.f || l != l ? (m - kShift + log2f(l)) * 0.69314718055994531f : -INFINITY;
          }
          tc_fence_before();                   // O is read before the next unit's products write it
        }
      }
    });
  } else if (warp < Z::kSoft + Z::kUnpack) {
    units([&]() {
      // ----------------------------------------------------------- unpack --
      const int tid = threadIdx.x - Z::kSoft * 32;
      const int token = tid % KT, g = tid / KT;    // a warp works on one group of its 32 tokens: its stores meet no bank twice
      const int32_t* table = P.page_table + static_cast<int64_t>(u.s) * P.ld_table;
      int lo0, hi0, lo1, hi1;                  // keys that some row of the unit sees
      sees(P, q, min(q.n - 1, rt * R / P.g), lo0, hi0);
      sees(P, q, min(q.n - 1, (rt * R + R - 1) / P.g), lo1, hi1);
      uint4 codes[2][2];
      uint32_t pairs[2];
      // the page of this thread's token in a tile (-1: not seen); loaded a tile before its codes are
      auto page_of = [&](int tile) {
        const int key = tile * KT + token;
        return key >= lo0 && key <= hi1 && tile < t0 + n_tiles ? __ldg(table + key / 16 / P.blocks_per_page) : -1;
      };
      auto block_of = [&](int tile, int id) -> const uint8_t* {
        const int key = tile * KT + token;
        if (key < lo0 || key > hi1) return nullptr;
        if (id < 0 || id >= P.c.n_pages) {
          if (P.c.status) atomicOr(P.c.status, kStatusPages);
          id = 0;
        }
        return P.c.pool + ((static_cast<int64_t>(id) * P.c.kv_heads + h) * P.blocks_per_page +
                           key / 16 % P.blocks_per_page) * (18 * D);
      };
      const int t = token % 16;
      auto fetch = [&](int kv, const uint8_t* blk) {       // codes and pair of this thread's 64 coordinates
        const uint8_t* src = blk + kv * 9 * D;
#pragma unroll
        for (int i = 0; i < 2; ++i)
          codes[kv][i] = blk ? __ldg(reinterpret_cast<const uint4*>(src + t * (D / 2) + g * 32) + i) : make_uint4(0, 0, 0, 0);
        pairs[kv] = blk ? __ldg(reinterpret_cast<const uint32_t*>(src + 8 * D + t * (D / 16)) + g) : 0u;
      };
      auto word = [&](int kv, int i) {
        const uint4 c4 = codes[kv][i / 4];
        return (i & 3) == 0 ? c4.x : (i & 3) == 1 ? c4.y : (i & 3) == 2 ? c4.z : c4.w;
      };
      const int row_at = g * (KT * 128) + token * 128, flip = (token % 8) * 16;
      auto put_k = [&]() {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&pairs[0]));
        // The high part's scale is at most 8188, so that 8 of it stay a binary16 number; what a larger one (up to 8736)
        // has beyond it is the remainder's: with the high part a multiple of 4, c s less it is one below 4400, 11 bits.
        const float top = fminf(f.x, 8188.f);
        const uint32_t s2 = pack_f16(f.x, f.x), top2 = pack_f16(top, top);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          uint32_t c[4], hi4[4], lo4[4];
          codes8<8>(word(0, i), c);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            hi4[e] = h2_mul(c[e], top2);
            lo4[e] = h2_fma(c[e], s2, hi4[e] ^ 0x80008000u);                // the product's exact remainder
          }
          uint8_t* to = sk + row_at + ((i * 16) ^ flip);
          *reinterpret_cast<uint4*>(to) = make_uint4(hi4[0], hi4[1], hi4[2], hi4[3]);
          *reinterpret_cast<uint4*>(to + Z::kKV) = make_uint4(lo4[0], lo4[1], lo4[2], lo4[3]);
        }
        // high, low, high part of z + 8 s against high, high, low of the sum of q
        const uint32_t hl = high_low(fmaf(8.f, f.x, f.y));
        *reinterpret_cast<uint16_t*>(skx + at_more(token, 3 * g)) = static_cast<uint16_t>(hl & 0xffffu);
        *reinterpret_cast<uint16_t*>(skx + at_more(token, 3 * g + 1)) = static_cast<uint16_t>(hl >> 16);
        *reinterpret_cast<uint16_t*>(skx + at_more(token, 3 * g + 2)) = static_cast<uint16_t>(hl & 0xffffu);
        fence_proxy_async_smem();
      };
      auto put_v = [&](uint32_t st) {
        uint32_t p = pairs[1];
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&p));
        const bool nan = f.x != f.x || f.y != f.y;
        const uint32_t nans = __ballot_sync(0xffffffffu, nan);
        if (lane == 0) lost[st * Z::kLost + g * (KT / 32) + token / 32] = nans;
        if (nan) p = 0;
        const uint32_t s2 = __byte_perm(p, p, 0x1010), z2 = __byte_perm(p, p, 0x3232);
        uint8_t* to = sv + st * Z::kKV + row_at;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          uint32_t c[4];
          codes8<0>(word(1, i), c);
          *reinterpret_cast<uint4*>(to + ((i * 16) ^ flip)) =
              make_uint4(h2_fma(c[0], s2, z2), h2_fma(c[1], s2, z2), h2_fma(c[2], s2, z2), h2_fma(c[3], s2, z2));
        }
        // z + 15 s may pass binary16's end (by 60, less than 2^-10 of it): its largest number then, in place of infinity
        if (fmaf(15.f, f.x, f.y) >= 65520.f) {
#pragma unroll 1
          for (int i = 0; i < 8; ++i) {
            uint4* at = reinterpret_cast<uint4*>(to + ((i * 16) ^ flip));
            const uint4 v = *at;
            constexpr uint32_t kEnd = 0x7bff7bffu;         // 65504
            *at = make_uint4(h2_min(v.x, kEnd), h2_min(v.y, kEnd), h2_min(v.z, kEnd), h2_min(v.w, kEnd));
          }
        }
        fence_proxy_async_smem();
      };
      const uint8_t* blk = nullptr;
      int id = -1;
      if (n_tiles > 0) {
        blk = block_of(t0, page_of(t0));
        fetch(0, blk);
        fetch(1, blk);
        id = page_of(t0 + 1);
      }
      for (int i = 0; i < n_tiles; ++i) {
        const uint32_t n = tiles_done + i, st = n & 1u;
        if (!(ok = wait_warp(k_free, n ^ 1u))) break;
        put_k();
        mbar_arrive(k_full);
        const bool next = i + 1 < n_tiles;
        if (next) {
          blk = block_of(t0 + i + 1, id);
          fetch(0, blk);                       // in flight while V is unpacked
          id = page_of(t0 + i + 2);
        }
        if (!(ok = wait_warp(v_free + st, (n >> 1) ^ 1u))) break;
        put_v(st);
        mbar_arrive(v_full + st);
        if (next) fetch(1, blk);
      }
    });
  } else {
    units([&]() {
      // -------------------------------------------------------- products --
      if (n_tiles > 0) {
        constexpr uint32_t kIdescS = idesc_f16_f32(128, KT);
        constexpr uint32_t kIdescO = idesc_f16_f32(128, D) | (1u << 16);      // B (V) is MN-major
        const uint32_t leader = elect_one();
        // descriptors of the operands; a step of 16 terms adds its bytes / 16
        const uint64_t d_q = smem_desc_sw128(smem_u32(sq), 1024), d_k = smem_desc_sw128(smem_u32(sk), 1024);
        const uint64_t d_qx = desc_plain16(smem_u32(sqx)), d_kx = desc_plain16(smem_u32(skx));
        const uint64_t d_v = desc_mn_sw128(smem_u32(sv), KT * 128);
        auto scores = [&](int qt) {
          const uint64_t dq = d_q + static_cast<uint32_t>(qt * (Z::kQ / 16));
          mma_ss(leader, tmem + qt * KT, d_qx + static_cast<uint32_t>(qt * (Z::kQx / 16)), d_kx, kIdescS, 0);
#pragma unroll
          for (int k = 0; k < D / 8; ++k) {    // the low parts, then the high ones
            const int kk = k % (D / 16);
            mma_ss(leader, tmem + qt * KT, dq + (kk / 4) * (128 * 128 / 16) + (kk % 4) * 2,
                   d_k + (k < D / 16 ? Z::kKV / 16 : 0) + (kk / 4) * (KT * 128 / 16) + (kk % 4) * 2, kIdescS, 1);
          }
          commit(leader, s_full + qt);
        };
        auto values = [&](int qt, uint32_t st, uint32_t more) {
          const uint64_t dv = d_v + st * (Z::kKV / 16);
#pragma unroll
          for (int k = 0; k < KT / 16; ++k)
            mma_ts(leader, tmem + Z::kO + qt * D, tmem + qt * KT + k * 8, dv + k * (2048 / 16), kIdescO, k > 0 ? 1u : more);
          commit(leader, o_done + qt);
        };
#pragma unroll 1
        for (int i = -1; i < n_tiles && ok; ++i) {
          const uint32_t n = tiles_done + i;   // the tile whose values are next; its scores are under way
          if (i >= 0) ok = wait_warp(v_full + (n & 1u), n >> 1);
#pragma unroll 1
          for (int qt = 0; qt < nqt && ok; ++qt) {
            const uint32_t tile = q_tiles_done[qt] + i;
            if (i < 0) {
              ok = wait_warp(q_full + qt, units_done[qt]);
              tc_fence_after();
            } else {
              if (!(ok = wait_warp(p_full + qt, tile))) break;
              tc_fence_after();
              values(qt, n & 1u, i > 0);
              if (qt == nqt - 1) commit(leader, v_free + (n & 1u));
              ok = wait_warp(o_done + qt, tile);           // the next scores go where these weights stand
            }
            if (ok && i + 1 < n_tiles) {
              // the keys are waited for here and not sooner: the first Q tile's values go on while they are unpacked
              if (qt == 0 && !(ok = wait_warp(k_full, n + 1))) break;
              tc_fence_after();
              scores(qt);
              if (qt == nqt - 1) commit(leader, k_free);
            }
          }
        }
        if (!ok) {                             // products in flight end before this warp goes on
          commit(leader, drain);
          mbar_wait(drain, 0, kDrainCycles);
        }
      }
    });
  }
  if (!ok && P.c.status) atomicOr(P.c.status, kStatusWait);
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == Z::kSoft + Z::kUnpack) tmem_dealloc(tmem, 512);
}

// Joins the partial sums of a unit that begins with worker w: a thread per row
// and 8 columns, the parts in order of the line.
template <int D, int R>
__global__ void __launch_bounds__(256) k_kv4_join_columns(const __grid_constant__ Params P) {
  const int w = blockIdx.x, tid = threadIdx.x;
  wait_for_stream();
  const int32_t* desc = P.desc + w * kDescInts;
  if (desc[0] != 1) return;
  const int q0 = desc[1], n = desc[2], h = desc[3], rt = desc[4], more = desc[5];
  const int row_in = blockIdx.y * 32 + tid % 32, row = rt * R + row_in;
  if (row >= n * P.g) return;
  auto part = [&](int i) {                     // slot 1 of worker w, then slot 0 of the ones behind it
    return P.partial + (static_cast<int64_t>(w + i) * 2 + (i == 0 ? 1 : 0)) * R * (D + 4) + row_in;
  };
  float m = kLowest, l = 0.f;
  for (int i = 0; i <= more; ++i) m = fmaxf(m, part(i)[D * R]);
  for (int i = 0; i <= more; ++i) l = fmaf(part(i)[(D + 1) * R], ex2(part(i)[D * R] - m), l);
  const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
  const int j = row / P.g, i0 = row - j * P.g;
  const int64_t orow = static_cast<int64_t>(q0 + j) * P.q_heads + h * P.g + i0;
  for (int c = (tid / 32) * 8; c < D; c += 64) {
    float o[8] = {};
    for (int i = 0; i <= more; ++i) {
      const float f = ex2(part(i)[D * R] - m) * inv;
#pragma unroll
      for (int k = 0; k < 8; ++k) o[k] = fmaf(part(i)[(c + k) * R], f, o[k]);
    }
    *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(P.out) + orow * D + c) =
        make_uint4(pack_bf16(o[0], o[1]), pack_bf16(o[2], o[3]), pack_bf16(o[4], o[5]), pack_bf16(o[6], o[7]));
  }
  if (tid < 32 && P.lse) P.lse[orow] = l > 0.f || l != l ? (m + log2f(l)) * 0.69314718055994531f : -INFINITY;
}

template <int D>
int run(Params& P, cudaStream_t st) {
  using Z = Shape<D>;
  static_assert(Z::kSmem <= 227 * 1024, "operands fit an SM");
  cudaError_t e = cudaFuncSetAttribute(k_kv4_prefill<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, Z::kSmem);
  if (e != cudaSuccess) return static_cast<int>(e);
  P.workers = kCtas;
  if (const int err = launch_dependent(k_kv4_prefill<D>, dim3(kCtas), dim3(Z::kThreads), Z::kSmem, st, P)) return err;
  return launch_dependent(k_kv4_join_columns<D, 128 * Z::QT>, dim3(P.workers, 4 * Z::QT), dim3(256), 0, st, P);
}

}  // namespace

size_t kv4_prefill_partial_bytes(int d) {
  return static_cast<size_t>(kCtas) * 2 * 128 * q_tiles_of(d) * (d + 4) * 4;
}

int launch_kv4_prefill(const Kv4Params& p, int d, void* stream) {
  Params P = p;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return d == 64 ? run<64>(P, st) : d == 128 ? run<128>(P, st) : run<256>(P, st);
}

}  // namespace tq
