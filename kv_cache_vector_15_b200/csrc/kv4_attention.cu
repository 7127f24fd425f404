// Attention of a few query rows over the paged 4-bit cache (decode, a handful
// of tokens at once, small cross attention).
//
// Mathematics.  With khat = z + s c (a pair per 64 coordinates), the logit is
//   <q, khat> = sum_g s_g <q_g, c_g> + z_g sum(q_g),
// an integer product per group of 64, so the codes go into the tensor cores as
// they are: unpacking 8 of them to bytes is two masks and a shift.  q is taken
// as 22-bit fixed-point numbers relative to the row's largest by a power of
// two, in three 8-bit limbs: a bf16 coordinate within 2^-13 of the largest is
// exact, any other is off by at most 2^-21 of it (two limbs, 2^-15, showed in
// the log-sum-exp); a group's sum of products, at most 64 * 15 * 2^21, fits 32
// bits.  fp32 rows have 30 bits in four limbs.  (mma.sync with e4m3 operands, which a byte 0..15 is too, measured 15 %
// slower: it is made of conversions and f16 products.)  Likewise
//   sum_t p_t vhat_t = sum_t (p_t s_t,g) c_t + sum_t p_t z_t,g,
// with p s in two bf16 terms (16 bits; one costs as much error as a bf16 output's
// rounding) against the code in the top bits of a bf16 mantissa: 16 + c for half
// of the tokens and, with the bits turned over, c - 31 for the others, so that
// the products stay balanced about zero (16 + c alone drove the sums of 131072
// tokens up and their truncation showed, 1.5e-3 of the output).  z - 16 s or
// z + 31 s goes in fp32 on the side.  fp32 rows: three terms, 24 bits, against
// c - 8, whose smaller products lose less; that takes a subtraction more per code
// (bf16 rows with it: 4 % more time).  Softmax keeps a
// running maximum and sum; the accumulators are rescaled only when a logit
// exceeds the maximum in use by 2^8 (any reference gives the same quotient).
//
// Bound: the packed bytes of K and V (18 d per 16 tokens and kv head).  The
// work per byte is issue slots, not tensor rate: keys stand on the M side of
// mma.sync (m16n8k32 u8 x s8, m16n8k16 bf16) and up to 4 query rows with
// their two terms fill its 8 columns, so nothing is padded, where a tcgen05
// tile would need 128 rows unpacked through shared memory for 4 to 16 query
// rows of use.  Every warp is a worker of its own with a ring of blocks in
// shared memory that it fills by bulk copies (one copy per 16-token block: K,
// V and their pairs are adjacent), so there is no block-wide barrier at all.
//
// Split: all blocks of all (sequence, kv head, row tile) units form one line
// that is cut into equal parts, one per warp, whatever the lengths are: the
// lengths stay on the device and a captured graph serves growing sequences.
// A unit that several warps share leaves partial sums, which a second kernel
// joins in order of the line (no atomics: the same inputs give the same bits).
//
// Measured, bf16, 8 kv heads of 4 query heads, d = 128: 8 x 131072 tokens
// 0.312 to 0.316 ms = 3.85 TB/s (59 % of the copy rate; the copies alone take 0.19 ms);
// 64 ragged sequences of 130 to 9000 tokens 65 to 67 us; one of 1000 12.1 us, the
// join included.  The schedulers issue in 54 % of their cycles, with 3 warps each,
// of which 0.92 can go on: it is independent work that is short, not slots.
// Warps wait for their own last results, for the ALU pipe (half rate,
// 51 % busy) or for instructions (the loop is 12 KB); 4 warps each need 128
// registers, spill, and take 0.341 ms.  One block a step 0.36, the next step's
// logits beside this one's values no gain; a third stage in the rings 0.002 slower.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <type_traits>

#include "kv4_internal.h"
#include "kv4_line.cuh"
#include "sm100.cuh"
#include "tq_internal.h"

namespace tq {
namespace {

using namespace sm100;

constexpr int kWarps = 4;                      // per CTA; each an independent worker
constexpr int kMaxWorkers = 148 * 16;
constexpr int kMinTiles = 4;                   // a worker's least share of the line: two steps
// What a unit costs besides its tiles (query rows, sums: about 9000 clocks), in tiles of 1800.  With 2, 5 and 9: 64
// sequences of 130 .. 9000 tokens 72.0, 64.5, 63.8 us, 256 of 100 .. 500 70.5, 67.2, 64.8, 16 of 1 .. 30000 60.8, 46.4,
// 38.0, 8 of 131072 309.5, 312.2, 313.4.
constexpr int kCost = 5;

// Blocks that a warp takes at a time, and stages of as many blocks in its ring.
__host__ __device__ constexpr int blocks_of(int d, int nt) { return d <= 128 && nt == 1 ? 2 : 1; }
__host__ __device__ constexpr int stages_of(int d, int nt) {
  return d == 64 ? 8 / blocks_of(d, nt) : d == 128 ? (nt == 1 ? 2 : 4) : 3;
}
// Column tiles of 4 rows that a unit has: as many as the largest sequence
// brings, up to two (d = 256: one, whose accumulators fill the registers).  One
// and two, 16 sequences of 8192 tokens, 8 kv heads, d = 128: 4 rows 53.2 and 76.8
// us, 8 rows 91 and 78, 16 rows 168 and 135 (a unit of two reads the cache once
// for 8 rows); d = 64 with 16384 tokens: 62 and 95, 110 and 96, 207 and 184.
constexpr int tiles_for(int d, int64_t rows) { return d == 256 || rows <= 4 ? 1 : 2; }
__host__ __device__ constexpr int ctas_of(int d, int nt) { return d <= 128 ? (nt == 1 ? 3 : 2) : 2; }

__device__ __forceinline__ float max_nan(float a, float b) {   // NaN where one is
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float from_bits_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float from_bits_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ void mma_u8s8(int (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k32.row.col.s32.u8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+r"(c[0]), "+r"(c[1]), "+r"(c[2]), "+r"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
// Two codes, at bits 0..3 and 16..19, to bf16 code - 8: 0x4300 | c is 128 + c.
__device__ __forceinline__ uint32_t centred(uint32_t w) {
  uint32_t t = (w & 0x000f000fu) | 0x43004300u, r;
  asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(t), "r"(0x43084308u));
  return r;
}

// Two codes, at bits 3..6 and 19..22, to bf16 16 + code, and to -(16 + 15 - code) = code - 31.
__device__ __forceinline__ uint32_t above16(uint32_t w) { return (w & 0x00780078u) | 0x41804180u; }
__device__ __forceinline__ uint32_t below16(uint32_t w) { return (~w & 0x00780078u) | 0xc180c180u; }

template <typename T>
__device__ __forceinline__ void load16(const T* p, float (&v)[16]);
template <>
__device__ __forceinline__ void load16<float>(const float* p, float (&v)[16]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float4 t = reinterpret_cast<const float4*>(p)[i];
    v[4 * i] = t.x; v[4 * i + 1] = t.y; v[4 * i + 2] = t.z; v[4 * i + 3] = t.w;
  }
}
template <>
__device__ __forceinline__ void load16<__nv_bfloat16>(const __nv_bfloat16* p, float (&v)[16]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint4 t = reinterpret_cast<const uint4*>(p)[i];
    const uint32_t w[4] = {t.x, t.y, t.z, t.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[8 * i + 2 * j] = from_bits_lo(w[j]);
      v[8 * i + 2 * j + 1] = from_bits_hi(w[j]);
    }
  }
}
template <typename T>
__device__ __forceinline__ void store8(T* p, const float (&v)[8]);
template <>
__device__ __forceinline__ void store8<float>(float* p, const float (&v)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
template <>
__device__ __forceinline__ void store8<__nv_bfloat16>(__nv_bfloat16* p, const float (&v)[8]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]),
                                            pack_bf16(v[6], v[7]));
}

// Lanes: r = lane / 4 and c = lane % 4.  A row of the logit tile is a token:
// row r stands for token r ^ ((r >> 1) & 1) of the block (and r + 8 likewise),
// an order in which the V reads of neighbouring lanes fall into both halves of
// the banks.  Column n of column tile t is query row 4 t + n % 4: in the logit
// product with its first limb for n < 4 and its second for n >= 4, then with the
// third and fourth (a column for each row and limb took 2 % more time than the
// exchange of four sums that this asks for); in the value product n < 4 has the
// first term of p s and n >= 4 the second.  A lane's accumulators are columns
// 2 c and 2 c + 1, so lanes c and c ^ 2 hold the two parts of the same query rows.
template <typename T, int D, int NT>
__global__ void __launch_bounds__(kWarps * 32, ctas_of(D, NT))
    k_kv4_decode(const __grid_constant__ Params P) {
  constexpr bool kF32 = sizeof(T) == 4;
  constexpr int G = D / 64;                    // groups of a row
  constexpr int NL = kF32 ? 4 : 3;             // limbs of a query coordinate
  constexpr uint32_t kBias = kF32 ? 0x80808080u : 0x808080u;
  constexpr int NB = blocks_of(D, NT);         // blocks of a step
  constexpr int R = 4 * NT;                    // query rows of a unit
  constexpr int BLK = 18 * D;                  // bytes of a block
  constexpr int NS = stages_of(D, NT);
  extern __shared__ __align__(16) uint8_t smem[];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, r = lane / 4, c = lane % 4;
  uint8_t* ring = smem + warp * NS * NB * BLK;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kWarps * NS * NB * BLK) + warp * NS;
  const int worker = blockIdx.x * kWarps + warp;
  wait_for_stream();
  if (worker >= P.workers) return;
  if (lane == 0) {
    for (int i = 0; i < NS; ++i) mbar_init(bars + i, 1);
    mbar_fence_init();
  }
  __syncwarp();

  const Part part = part_of<16, kCost>(P, worker, R, kMinTiles);
  int32_t* desc = P.desc + worker * kDescInts;
  if (lane == 0) desc[0] = 0;                  // no unit begins here that others go on with
  if (part.a >= part.b) return;
  Piece u = piece_at(part);
  if (!settle<16, kCost>(P, R, part.b, u)) return;

  uint32_t phases = 0;                         // parity of each stage's barrier
  bool ok = true;
  // The copies' own place in the piece: page ids of the next 32 pages, one per
  // lane, and the next block.
  const int32_t* table = nullptr;
  int page_i = 0, blk = 0, page_base = 0, last_page = 0, ids = 0;
  auto refill = [&]() {
    page_base = page_i;
    const int pi = page_i + lane;
    ids = pi <= last_page ? table[pi] : 0;
    if (ids < 0 || ids >= P.c.n_pages) {
      if (P.c.status) atomicOr(P.c.status, kStatusPages);
      ids = 0;
    }
  };
  auto issue = [&](int stage, int left) {      // whole warp; the next blocks in order
    if (lane == 0) mbar_arrive_expect_tx(bars + stage, min(left, NB) * BLK);
#pragma unroll
    for (int bk = 0; bk < NB; ++bk) {
      if (bk < left) {
        if (page_i - page_base >= 32) refill();
        const int id = __shfl_sync(0xffffffffu, ids, page_i - page_base);
        if (lane == 0)
          bulk_load(ring + (stage * NB + bk) * BLK,
                    P.c.pool + ((static_cast<int64_t>(id) * P.c.kv_heads + u.h) * P.blocks_per_page + blk) * BLK, BLK,
                    bars + stage);
        if (++blk == P.blocks_per_page) {
          blk = 0;
          ++page_i;
        }
      }
    }
  };
  auto begin_copies = [&]() {                  // of the piece, into the first stages
    if (u.n_tiles == 0) return;
    table = P.page_table + static_cast<int64_t>(u.s) * P.ld_table;
    page_i = u.t0 / P.blocks_per_page;
    blk = u.t0 - page_i * P.blocks_per_page;
    last_page = (u.t0 + u.n_tiles - 1) / P.blocks_per_page;
    refill();
    for (int i = 0; i < NS && i * NB < u.n_tiles; ++i) issue(i, u.n_tiles - i * NB);
  };
  begin_copies();

  for (bool more = true; more;) {
    const Seq q = u.q;
    const int h = u.h, rt = u.rt, t0 = u.t0, n_tiles = u.n_tiles;

    // query rows as limbs (high, middle, low): B operands of the logit product
    uint32_t qb[NT][2][2 * G][2];              // [high | middle, low | next][step of 32 coordinates][register]
    float qscale[NT][2], qsum[NT][G][2];       // logit = qscale (s (limbs . c) + z qsum); qsum in lanes c >= 2 only
    int lo[NT][2], hi[NT][2];
    int full_lo = 0, full_hi = 0x7fffffff;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int row = rt * R + 4 * t + (r & 3), n_rows = q.n * P.g;
      const bool live = row < n_rows;
      const int j = live ? row / P.g : 0, i = row - j * P.g;
      const T* src = static_cast<const T*>(P.q) + (q.q0 + j) * P.ld_q + static_cast<int64_t>(h * P.g + i) * D + 16 * c;
      int lo1, hi1;
      sees(P, q, live ? j : q.n - 1, lo1, hi1);
      full_lo = max(full_lo, lo1);
      full_hi = min(full_hi, hi1);
      float v[G][16], top = 0.f;
#pragma unroll
      for (int g = 0; g < G; ++g) {
        if (live) {
          load16(src + 64 * g, v[g]);
        } else {
#pragma unroll
          for (int e = 0; e < 16; ++e) v[g][e] = 0.f;
        }
#pragma unroll
        for (int e = 0; e < 16; ++e) top = fmaxf(top, fabsf(v[g][e]));
      }
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      // 2^ex such that top 2^ex <= 2^21 (fp32 rows: 2^29)
      int ex = 0;
      frexpf(top, &ex);
      ex = top > 0.f ? min((kF32 ? 29 : 21) - ex, 120) : 0;
      // an infinite coordinate: its logits are infinite or NaN, and NaN the softmax of such (a NaN comes in by the sums)
      const float up = pow2(ex), down = top < INFINITY ? P.scale_log2 * pow2(-ex) : __int_as_float(0x7fffffff);
#pragma unroll
      for (int g = 0; g < G; ++g) {
        float sum = 0.f;
        uint32_t w[NL][4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {          // word k / 2; its even coordinates are k 0..15 of a step, its odd ones k 16..31
          uint32_t x[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float f = v[g][(k / 2) * 8 + 2 * e + (k & 1)] * up;
            sum += f;
            // a number in digits of base 256 in [-128, 127]: adding 128 to each makes them the bytes of a number, and
            // flipping the bytes' top bits takes it off again
            x[e] = (static_cast<uint32_t>(__float2int_rn(f)) + kBias) ^ kBias;
          }
          const uint32_t a01 = __byte_perm(x[0], x[1], 0x5140), a23 = __byte_perm(x[2], x[3], 0x5140);
          const uint32_t b01 = __byte_perm(x[0], x[1], 0x7362), b23 = __byte_perm(x[2], x[3], 0x7362);
          w[NL - 1][k] = __byte_perm(a01, a23, 0x5410);
          w[NL - 2][k] = __byte_perm(a01, a23, 0x7632);
          w[NL - 3][k] = __byte_perm(b01, b23, 0x5410);
          if (kF32) w[0][k] = __byte_perm(b01, b23, 0x7632);
        }
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
          for (int i = 0; i < 2; ++i) {        // columns 4..7 have the second limb of each two
            qb[t][0][2 * g + k][i] = r < 4 ? w[0][2 * k + i] : w[1][2 * k + i];
            qb[t][1][2 * g + k][i] = r < 4 ? w[2][2 * k + i] : kF32 ? w[NL - 1][2 * k + i] : 0u;
          }
#pragma unroll
        for (int k = 0; k < 2; ++k) {          // of the two query rows in this lane's columns
          const float of = __shfl_sync(0xffffffffu, sum, ((2 * c + k) & 3) * 4);
          qsum[t][g][k] = c >= 2 ? of : 0.f;
        }
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) qscale[t][k] = __shfl_sync(0xffffffffu, down, ((2 * c + k) & 3) * 4);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int from = ((2 * c + k) & 3) * 4;
        lo[t][k] = __shfl_sync(0xffffffffu, lo1, from);
        hi[t][k] = __shfl_sync(0xffffffffu, hi1, from);
      }
    }
#pragma unroll
    for (int o = 4; o < 16; o <<= 1) {         // lanes r & 3 hold the rows of each column tile
      full_lo = max(full_lo, __shfl_xor_sync(0xffffffffu, full_lo, o));
      full_hi = min(full_hi, __shfl_xor_sync(0xffffffffu, full_hi, o));
    }

    float acc[NT][D / 16][4], zacc[NT][G][2], mx[NT][2], den[NT][2];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) acc[t][i][k] = 0.f;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        mx[t][k] = kLowest;
        den[t][k] = 0.f;
#pragma unroll
        for (int g = 0; g < G; ++g) zacc[t][g][k] = 0.f;
      }
    }

    const int tr = r ^ ((r >> 1) & 1);         // token of row r; r + 8: tr + 8
    const float low_term = c >= 2 ? 1.f : 0.f;
    const int first_limb = c >= 2 ? 256 : 65536;
    const int key_end = (t0 + n_tiles) * 16;   // what follows is another worker's, or not loaded
    // NB blocks of 16 tokens; kEdge: some of these tokens are not seen by some row, or not there.
    auto step = [&](auto edge, const uint8_t* blocks, int key0) {
      constexpr bool kEdge = decltype(edge)::value;
      float sc[NB][NT][4];

      // ---- logits ---------------------------------------------------------
#pragma unroll
      for (int bg = 0; bg < NB * G; ++bg) {
        const int bk = bg / G, g = bg % G;
        const uint8_t* kc = blocks + bk * BLK;
        const uint2 w0 = *reinterpret_cast<const uint2*>(kc + tr * (D / 2) + 32 * g + 8 * c);
        const uint2 w1 = *reinterpret_cast<const uint2*>(kc + (tr + 8) * (D / 2) + 32 * g + 8 * c);
        const uint32_t p0 = *reinterpret_cast<const uint32_t*>(kc + 8 * D + tr * (D / 16) + 4 * g);
        const uint32_t p1 = *reinterpret_cast<const uint32_t*>(kc + 8 * D + (tr + 8) * (D / 16) + 4 * g);
        const float2 f0 = __half22float2(*reinterpret_cast<const __half2*>(&p0));
        const float2 f1 = __half22float2(*reinterpret_cast<const __half2*>(&p1));
        const uint32_t A[2][4] = {
            {w0.x & 0x0f0f0f0fu, w1.x & 0x0f0f0f0fu, (w0.x >> 4) & 0x0f0f0f0fu, (w1.x >> 4) & 0x0f0f0f0fu},
            {w0.y & 0x0f0f0f0fu, w1.y & 0x0f0f0f0fu, (w0.y >> 4) & 0x0f0f0f0fu, (w1.y >> 4) & 0x0f0f0f0fu}};
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          int x[2][4] = {};
#pragma unroll
          for (int l = 0; l < 2; ++l)
#pragma unroll
            for (int k = 0; k < 2; ++k) mma_u8s8(x[l], A[k], qb[t][l][2 * g + k][0], qb[t][l][2 * g + k][1]);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float2 pair = k < 2 ? f0 : f1;
            const float f = kF32 ? fmaf(static_cast<float>(x[0][k]), 65536.f, static_cast<float>(x[1][k]))
                                 : static_cast<float>(x[0][k] * first_limb + x[1][k]);
            const float z = g == 0 ? pair.y * qsum[t][g][k & 1] : fmaf(pair.y, qsum[t][g][k & 1], sc[bk][t][k]);
            sc[bk][t][k] = fmaf(pair.x, f, z);
          }
        }
      }

      // the limbs in columns 0..3 and those in columns 4..7 (with the zeros' term) add up
#pragma unroll
      for (int bk = 0; bk < NB; ++bk)
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if (kF32) sc[bk][t][k] *= c >= 2 ? 1.f : 256.f;
            sc[bk][t][k] += __shfl_xor_sync(0xffffffffu, sc[bk][t][k], 2);
          }

      // ---- softmax --------------------------------------------------------
      // an edge's logits are scaled and masked first; the others' scale goes into the subtraction of the maximum
      if (kEdge) {
#pragma unroll
        for (int bk = 0; bk < NB; ++bk)
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int key = key0 + 16 * bk + tr + (k < 2 ? 0 : 8);
              sc[bk][t][k] *= qscale[t][k & 1];
              if (key < lo[t][k & 1] || key > hi[t][k & 1] || key >= key_end) sc[bk][t][k] = -INFINITY;
            }
      }
      auto factor = [&](int t, int k) { return kEdge ? 1.f : qscale[t][k & 1]; };
      float top = -INFINITY, y[NB][NT][4];
#pragma unroll
      for (int bk = 0; bk < NB; ++bk)
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            y[bk][t][k] = fmaf(sc[bk][t][k], factor(t, k), -mx[t][k & 1]);
            top = fmaxf(top, y[bk][t][k]);
          }
      if (__any_sync(0xffffffffu, top > kLazy)) {
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            float m = mx[t][k];
#pragma unroll
            for (int bk = 0; bk < NB; ++bk)
              m = fmaxf(m, fmaxf(sc[bk][t][k] * factor(t, k), sc[bk][t][k + 2] * factor(t, k)));
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 4));
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 8));
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
            const float f = ex2(mx[t][k] - m);
            mx[t][k] = m;
            den[t][k] *= f;
#pragma unroll
            for (int g = 0; g < G; ++g) zacc[t][g][k] *= f;
#pragma unroll
            for (int j = 0; j < D / 16; ++j) {
              acc[t][j][k] *= f;
              acc[t][j][k + 2] *= f;
            }
#pragma unroll
            for (int bk = 0; bk < NB; ++bk) {
              y[bk][t][k] = fmaf(sc[bk][t][k], factor(t, k), -m);
              y[bk][t][k + 2] = fmaf(sc[bk][t][k + 2], factor(t, k), -m);
            }
          }
      }
#pragma unroll
      for (int bk = 0; bk < NB; ++bk)
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            sc[bk][t][k] = ex2(y[bk][t][k]);
            // at an edge a weight of zero stands for a token that is not seen: a seen one's is not less than 2^-126 (a
            // part of 2^-118 of the sum at most), so that a NaN value behind it counts here as it does elsewhere
            if (kEdge && y[bk][t][k] != -INFINITY) sc[bk][t][k] = max_nan(sc[bk][t][k], 1.17549435e-38f);
            den[t][k & 1] += sc[bk][t][k];
          }

      // ---- values ---------------------------------------------------------
#pragma unroll
      for (int bg = 0; bg < NB * G; ++bg) {
        const int bk = bg / G, g = bg % G;
        const uint8_t* vc = blocks + bk * BLK + 9 * D;
        const uint32_t p0 = *reinterpret_cast<const uint32_t*>(vc + 8 * D + tr * (D / 16) + 4 * g);
        const uint32_t p1 = *reinterpret_cast<const uint32_t*>(vc + 8 * D + (tr + 8) * (D / 16) + 4 * g);
        const float2 f0 = __half22float2(*reinterpret_cast<const __half2*>(&p0));
        const float2 f1 = __half22float2(*reinterpret_cast<const __half2*>(&p1));
        // the codes enter as c - 8, or as 16 + c (the first 8 tokens) and c - 31 (the others)
        const float z0 = fmaf(kF32 ? 8.f : -16.f, f0.x, f0.y), z1 = fmaf(kF32 ? 8.f : 31.f, f1.x, f1.y);
        uint32_t pb[NT][2], pb3[kF32 ? NT : 1][2];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          float x[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            x[k] = sc[bk][t][k] * (k < 2 ? f0.x : f1.x);
            float z = k < 2 ? z0 : z1;
            if (kEdge && sc[bk][t][k] == 0.f) {  // a token that is not seen: whatever its bytes stand for
              x[k] = 0.f;
              z = 0.f;
            }
            zacc[t][g][k & 1] = fmaf(sc[bk][t][k], z, zacc[t][g][k & 1]);
          }
#pragma unroll
          for (int k = 0; k < 2; ++k) {        // lanes c < 2 the first term of p s, the others the second
            const uint32_t u = pack_bf16(x[2 * k], x[2 * k + 1]);
            const float y0 = fmaf(-low_term, from_bits_lo(u), x[2 * k]), y1 = fmaf(-low_term, from_bits_hi(u), x[2 * k + 1]);
            const uint32_t w = pack_bf16(y0, y1);
            pb[t][k] = transpose8x8(w);
            if (kF32)                          // the third term, in the columns of the second
              pb3[kF32 ? t : 0][k] = transpose8x8(pack_bf16(low_term * (y0 - from_bits_lo(w)), low_term * (y1 - from_bits_hi(w))));
          }
        }
        // tokens of k = 2c, 2c+1, 2c+8, 2c+9, coordinates 64 g + 8 r + 0..7
        const int ta = (2 * c) ^ (c & 1), tb = (2 * c + 1) ^ (c & 1);
        const uint8_t* vr = vc + 32 * g + 4 * r;
        const uint32_t wa = *reinterpret_cast<const uint32_t*>(vr + ta * (D / 2));
        const uint32_t wb = *reinterpret_cast<const uint32_t*>(vr + tb * (D / 2));
        const uint32_t wc = *reinterpret_cast<const uint32_t*>(vr + (ta + 8) * (D / 2));
        const uint32_t wd = *reinterpret_cast<const uint32_t*>(vr + (tb + 8) * (D / 2));
        const uint32_t u[2] = {__byte_perm(wa, wb, 0x5410), __byte_perm(wa, wb, 0x7632)};
        const uint32_t v[2] = {__byte_perm(wc, wd, 0x5410), __byte_perm(wc, wd, 0x7632)};
#pragma unroll
        for (int j = 0; j < 4; ++j) {          // rows of the tile: coordinates 8 r + 2 j and 8 r + 2 j + 1
          uint32_t a0, a1, a2, a3;
          if constexpr (kF32) {
            a0 = centred(u[j / 2] >> (8 * (j & 1)));
            a1 = centred(u[j / 2] >> (8 * (j & 1) + 4));
            a2 = centred(v[j / 2] >> (8 * (j & 1)));
            a3 = centred(v[j / 2] >> (8 * (j & 1) + 4));
          } else {
            a0 = above16(j & 1 ? u[j / 2] >> 5 : u[j / 2] << 3);
            a1 = above16(u[j / 2] >> (8 * (j & 1) + 1));
            a2 = below16(j & 1 ? v[j / 2] >> 5 : v[j / 2] << 3);
            a3 = below16(v[j / 2] >> (8 * (j & 1) + 1));
          }
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            mma_bf16(acc[t][4 * g + j], a0, a1, a2, a3, pb[t][0], pb[t][1]);
            if (kF32) mma_bf16(acc[t][4 * g + j], a0, a1, a2, a3, pb3[kF32 ? t : 0][0], pb3[kF32 ? t : 0][1]);
          }
        }
      }
    };

    int stage = 0, i = 0;
    for (; i < n_tiles; i += NB) {
      ok = mbar_wait(bars + stage, (phases >> stage) & 1u, P.limit);
      if (!__all_sync(0xffffffffu, ok)) {
        ok = false;
        break;
      }
      phases ^= 1u << stage;
      const int key0 = (t0 + i) * 16;
      if (key0 < full_lo || key0 + 16 * NB - 1 > full_hi || i + NB > n_tiles)
        step(std::true_type{}, ring + stage * NB * BLK, key0);
      else
        step(std::false_type{}, ring + stage * NB * BLK, key0);
      __syncwarp();                            // every lane has read the stage
      if (i + NS * NB < n_tiles) issue(stage, n_tiles - (i + NS * NB));
      stage = stage + 1 == NS ? 0 : stage + 1;
    }
    if (!ok) {
      // a copy did not arrive in time: record it, and wait for those still in flight before the ring goes
      for (int k = 0; k < NS && i + k * NB < n_tiles; ++k) {
        const int st = (stage + k) % NS;
        mbar_wait(bars + st, (phases >> st) & 1u, kDrainCycles);
      }
      if (lane == 0 && P.c.status) atomicOr(P.c.status, kStatusWait);
      break;
    }

    // ---- the unit's sums, while the next piece's copies are under way --------
    const bool whole = u.whole, first = u.first;
    if (!whole && first && lane == 0) describe(desc, u, part.share, worker);
    more = next_piece<16, kCost>(P, R, part.b, u);
    if (more) begin_copies();
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) {
          den[t][k] += __shfl_xor_sync(0xffffffffu, den[t][k], o);
#pragma unroll
          for (int g = 0; g < G; ++g) zacc[t][g][k] += __shfl_xor_sync(0xffffffffu, zacc[t][g][k], o);
        }
      }
      const int k = c >= 2 ? 1 : 0;            // lanes c and c ^ 2 write one of their two query rows each
      const int row_in = 4 * t + 2 * (c & 1) + k, row = rt * R + row_in;
      const float l = k ? den[t][1] : den[t][0], m = k ? mx[t][1] : mx[t][0];
      const float inv = whole ? (l > 0.f || l != l ? 1.f / l : 0.f) : 1.f;
      const int j = row / P.g, i = row - j * P.g;
      const int64_t orow = static_cast<int64_t>(q.q0 + j) * P.q_heads + h * P.g + i;
      float* sums = P.partial + (static_cast<int64_t>(worker) * 2 + (first ? 1 : 0)) * R * (D + 4) +
                    row_in * (D + 4);
      const bool live = row < q.n * P.g;
#pragma unroll
      for (int g = 0; g < G; ++g) {
        float o[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float* x = acc[t][4 * g + e];
          const float s0 = x[0] + __shfl_xor_sync(0xffffffffu, x[0], 2), s1 = x[1] + __shfl_xor_sync(0xffffffffu, x[1], 2);
          const float s2 = x[2] + __shfl_xor_sync(0xffffffffu, x[2], 2), s3 = x[3] + __shfl_xor_sync(0xffffffffu, x[3], 2);
          const float z = k ? zacc[t][g][1] : zacc[t][g][0];
          o[2 * e] = ((k ? s1 : s0) + z) * inv;
          o[2 * e + 1] = ((k ? s3 : s2) + z) * inv;
        }
        if (whole) {
          if (live) store8(static_cast<T*>(P.out) + orow * D + 64 * g + 8 * r, o);
        } else {
          store8(sums + 64 * g + 8 * r, o);
        }
      }
      if (r == 0) {
        if (!whole) {
          sums[D] = m;
          sums[D + 1] = l;
        } else if (live && P.lse) {
          P.lse[orow] = l > 0.f || l != l ? (m + log2f(l)) * 0.69314718055994531f : -INFINITY;
        }
      }
    }
  }
}

// Joins the partial sums of units that several workers share, the parts in
// order of the line.  CTA (x, row): the units that begin with one of the
// workers x, x + gridDim.x, ...; its warps take quarters of a unit's parts.
template <typename T, int D, int R>
__global__ void __launch_bounds__(128) k_kv4_join(const __grid_constant__ Params P) {
  constexpr int E = D / 32;
  __shared__ float sums[4][D + 2];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, row_in = blockIdx.y;
  wait_for_stream();
  for (int w0 = blockIdx.x; w0 < P.workers; w0 += 32 * gridDim.x) {
    const int mine = w0 + lane * gridDim.x;
    uint32_t found = __ballot_sync(0xffffffffu, mine < P.workers && P.desc[mine * kDescInts] == 1);
    for (; found; found &= found - 1) {        // the same for every warp
      const int w = w0 + (__ffs(found) - 1) * gridDim.x;
      const int32_t* desc = P.desc + w * kDescInts;
      const int q0 = desc[1], n = desc[2], h = desc[3], rt = desc[4], parts = desc[5] + 1;
      const int row = rt * R + row_in;
      if (row >= n * P.g) continue;
      // slot 1 of worker w, then slot 0 of the ones behind it
      auto part = [&](int i) {
        return P.partial + (static_cast<int64_t>(w + i) * 2 + (i == 0 ? 1 : 0)) * R * (D + 4) + row_in * (D + 4);
      };
      const int per = (parts + 3) / 4, i0 = warp * per, i1 = min(i0 + per, parts);
      float m = kLowest;
      for (int i = i0 + lane; i < i1; i += 32) m = fmaxf(m, part(i)[D]);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      float l = 0.f, o[E];
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] = 0.f;
#pragma unroll 4
      for (int i = i0; i < i1; ++i) {
        const float* p = part(i);
        const float f = ex2(p[D] - m);
        l = fmaf(p[D + 1], f, l);
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = fmaf(p[lane * E + e], f, o[e]);
      }
      __syncthreads();                         // sums of a unit before this one are read
#pragma unroll
      for (int e = 0; e < E; ++e) sums[warp][lane * E + e] = o[e];
      if (lane == 0) {
        sums[warp][D] = m;
        sums[warp][D + 1] = l;
      }
      __syncthreads();
      m = fmaxf(fmaxf(sums[0][D], sums[1][D]), fmaxf(sums[2][D], sums[3][D]));
      float f[4];
      l = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        f[i] = ex2(sums[i][D] - m);
        l = fmaf(sums[i][D + 1], f[i], l);
      }
      const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
      const int j = row / P.g, hh = row - j * P.g;
      const int64_t orow = static_cast<int64_t>(q0 + j) * P.q_heads + h * P.g + hh;
      for (int e = threadIdx.x; e < D; e += 128) {
        float x = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) x = fmaf(sums[i][e], f[i], x);
        if constexpr (sizeof(T) == 4) static_cast<T*>(P.out)[orow * D + e] = x * inv;
        else static_cast<T*>(P.out)[orow * D + e] = __float2bfloat16_rn(x * inv);
      }
      if (threadIdx.x == 0 && P.lse) P.lse[orow] = l > 0.f || l != l ? (m + log2f(l)) * 0.69314718055994531f : -INFINITY;
    }
  }
}

template <typename T, int D, int NT>
int run(Params& P, cudaStream_t st) {
  constexpr int smem = kWarps * stages_of(D, NT) * (blocks_of(D, NT) * 18 * D + 8);
  static_assert(smem <= 227 * 1024, "the rings fit an SM");
  cudaError_t e = cudaSuccess;
  if (smem > 48 * 1024) {
    e = cudaFuncSetAttribute(k_kv4_decode<T, D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return static_cast<int>(e);
  }
  constexpr int per_sm = ctas_of(D, NT);
  P.workers = 148 * per_sm * kWarps;
  if (const int err = launch_dependent(k_kv4_decode<T, D, NT>, dim3(148 * per_sm), dim3(kWarps * 32), smem, st, P)) return err;
  return launch_dependent(k_kv4_join<T, D, 4 * NT>, dim3(148, 4 * NT), dim3(128), 0, st, P);
}

template <typename T>
int run_d(Params& P, int d, int rows, cudaStream_t st) {
  const int nt = tiles_for(d, rows);
  if (d == 64) return nt == 1 ? run<T, 64, 1>(P, st) : run<T, 64, 2>(P, st);
  if (d == 128) return nt == 1 ? run<T, 128, 1>(P, st) : run<T, 128, 2>(P, st);
  return run<T, 256, 1>(P, st);
}

}  // namespace

// bf16 rows go to the kernel for many rows from 17 rows per kv head on: below,
// its tiles of 128 rows are mostly empty.  This kernel and that one, 16 sequences
// of 8192 tokens, 8 kv heads, d = 128: 16 rows 135 and 182 us, 20 rows 191 and
// 184, 64 rows 487 and 187; d = 64, 16384 tokens: 184 and 264, 275 and 264; d =
// 256, 4 kv heads: 166 and 184, 203 and 186.  (Short caches cross later: 4
// sequences of 1000 tokens, 20 rows 20.5 and 27.9 us, 64 rows 31 and 31.)  fp32
// rows stay here whatever their number: that kernel's query operands have the
// 11 bits of binary16.
bool kv4_prefill_applies(int bf16, int64_t rows) { return bf16 && rows > 16; }

size_t kv4_attention_ws_bytes(int d, int bf16, int64_t rows) {
  const size_t desc = round256(static_cast<size_t>(kMaxWorkers) * kDescInts * 4);
  if (kv4_prefill_applies(bf16, rows)) return desc + kv4_prefill_partial_bytes(d);
  return desc + static_cast<size_t>(148) * ctas_of(d, tiles_for(d, rows)) * kWarps * 2 * 4 * tiles_for(d, rows) * (d + 4) * 4;
}

int launch_kv4_attention(const Kv4Attn& a, int bf16, void* stream) {
  if (take_injected_launch_failure()) return static_cast<int>(cudaErrorLaunchFailure);
  Params P;
  P.c = a.c;
  P.q = a.q;
  P.ld_q = a.ld_q;
  P.n_tokens = a.n_tokens;
  P.ld_table = a.ld_table;
  P.q_heads = a.q_heads;
  P.g = a.q_heads / a.c.kv_heads;
  P.n_seqs = a.n_seqs;
  P.blocks_per_page = a.c.page_size / 16;
  P.cu_q = a.cu_q;
  P.page_table = a.page_table;
  P.seq_lens = a.seq_lens;
  P.scale_log2 = a.scale * 1.44269504088896341f;
  P.causal = a.causal;
  P.window = a.window;
  P.out = a.out;
  P.lse = a.lse;
  P.desc = static_cast<int32_t*>(a.ws);
  P.partial = reinterpret_cast<float*>(static_cast<uint8_t*>(a.ws) +
                                       round256(static_cast<size_t>(kMaxWorkers) * kDescInts * 4));
  P.limit = wait_limit_cycles();
  P.workers = 0;
  const int64_t rows = static_cast<int64_t>(a.max_q) * P.g;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int r = static_cast<int>(std::min<int64_t>(rows, 1 << 20));
  if (kv4_prefill_applies(bf16, rows)) return launch_kv4_prefill(P, a.c.d, stream);
  return bf16 ? run_d<__nv_bfloat16>(P, a.c.d, r, st) : run_d<float>(P, a.c.d, r, st);
}

}  // namespace tq
