// The paged 4-bit cache's write and read back: rows of k and v to codes and
// (scale, zero) pairs in their slots, and the values they stand for.
//
// Bound: bytes.  An appended bf16 row moves 2 d bytes in and 9 d / 16 out (and
// 2 d more where the values are wanted).  A thread takes 16 coordinates of a
// row (two 16-byte loads of bf16, four of fp32), so a group of 64 is 4
// neighbouring lanes: its minimum and maximum are 2 shuffles each, its codes
// one 8-byte store per lane, and all that is kept is in registers.  What bounds
// it in practice is issue slots (taken in 73 % of the cycles) and the loads that
// are in flight.  32768 tokens
// of 8 heads, d = 128, bf16, with values (306 MB): 8 coordinates a thread 90 us,
// in which the quotients, addresses and conversions of a group weigh more; 16
// with 63 registers 83 us, with 40 registers (the coordinates are read again
// where fp64 has to decide) 72 us, 4.25 TB/s; fp32 rows, 574 MB in all, 102 us,
// 5.6 TB/s.
//
// The code is rint((x - z) / s) with the exact quotient, so that every form of
// the cache agrees on every bit.  fp32 decides it where the fp32 value of the
// quotient is further from a border than its error: (x - z), 1 / (15 s), their
// product and its product with 15 are each off by at most 2^-24 of at most 16,
// 4e-6 in all, so a thread that has a quotient within 1e-5 of a border
// compares x with the border z + (k + 1/2) s in fp64, in which that is exact
// (x - z is not, for an x far smaller than z).  Otherwise the
// clamp to [0, 15] is the product's saturation, and the rounding an addition
// of 1.5 * 2^23 whose low bits are the code: 7 instructions a coordinate.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "kv4_internal.h"
#include "launch.cuh"
#include "tq_internal.h"

namespace tq {
namespace {

constexpr int kThreads = 256;

// Sixteen neighbouring coordinates as they were loaded, and as numbers.
template <typename T>
struct Sixteen;
template <>
struct Sixteen<float> {
  float4 t[4];
  __device__ __forceinline__ void load(const float* p) {
#pragma unroll
    for (int i = 0; i < 4; ++i) t[i] = __ldcs(reinterpret_cast<const float4*>(p) + i);
  }
  __device__ __forceinline__ void get(float (&v)[16]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[4 * i] = t[i].x; v[4 * i + 1] = t[i].y; v[4 * i + 2] = t[i].z; v[4 * i + 3] = t[i].w;
    }
  }
};
template <>
struct Sixteen<__nv_bfloat16> {
  uint4 t[2];
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    t[0] = __ldcs(reinterpret_cast<const uint4*>(p));
    t[1] = __ldcs(reinterpret_cast<const uint4*>(p) + 1);
  }
  __device__ __forceinline__ void get(float (&v)[16]) const {
    const uint32_t w[8] = {t[0].x, t[0].y, t[0].z, t[0].w, t[1].x, t[1].y, t[1].z, t[1].w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
};
template <typename T>
__device__ __forceinline__ void store8(T* p, const float (&v)[8]);
template <>
__device__ __forceinline__ void store8<float>(float* p, const float (&v)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
template <>
__device__ __forceinline__ void store8<__nv_bfloat16>(__nv_bfloat16* p, const float (&v)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    __nv_bfloat162 t = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    w[i] = *reinterpret_cast<uint32_t*>(&t);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

// The smaller, the larger; NaN where one is.
__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// What the host works out once per call.
struct Sizes {
  int64_t n_slots;                     // of the pool
  double inv_ps;                       // 1 / page_size
  uint32_t page_bytes;                 // less than 2^31 for every size that the format has
  int head_bytes, log_chunks, units;   // units of a token: 2 kv_heads d / 16
};
// Bytes from the pool's begin to a slot's 16-token block of kv head 0, and the token's place in it.
__device__ __forceinline__ int64_t block_of(const tq_kv4& c, const Sizes& z, int64_t slot, int& t) {
  // slot / page_size (slot < 2^42): the fp64 product is off by less than one
  int page = static_cast<int>(static_cast<double>(slot) * z.inv_ps);
  int rest = static_cast<int>(slot - static_cast<int64_t>(page) * c.page_size);
  if (rest < 0) {
    --page;
    rest += c.page_size;
  } else if (rest >= c.page_size) {
    ++page;
    rest -= c.page_size;
  }
  t = rest & 15;
  return static_cast<int64_t>(static_cast<uint64_t>(page) * z.page_bytes) + (rest >> 4) * (18 * c.d);
}

// A unit is 16 coordinates of one row: chunk, part (K or V) and head are bits of
// its number within the token, so nothing is divided; threadIdx.y counts tokens.
struct Unit {
  int chunk, part, h;
};
__device__ __forceinline__ Unit unit_of(int u, int log_chunks) {
  return {u & ((1 << log_chunks) - 1), (u >> log_chunks) & 1, u >> (log_chunks + 1)};
}

template <typename T>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 ? 6 : 5) k_kv4_append(tq_kv4 c, const T* k, int64_t ld_k, const T* v, int64_t ld_v,
                                                            int64_t n_tokens, const int64_t* slots, T* kv, T* vv,
                                                            Sizes z) {
  wait_for_stream();
  const int64_t token_at = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y;
  const bool live = token_at < n_tokens;                  // a warp may hold tokens of both kinds: its shuffles need all
  const int64_t token = live ? token_at : n_tokens - 1;
  const int64_t slot = slots[token];
  const bool stored = live && slot >= 0 && slot < z.n_slots;
  if (live && slot >= z.n_slots && threadIdx.x == 0 && blockIdx.y == 0 && c.status) atomicOr(c.status, kStatusIndex);
  int t;
  uint8_t* block = c.pool + block_of(c, z, stored ? slot : 0, t);
  k += token * ld_k;
  v += token * ld_v;
  const int64_t row0 = token * c.kv_heads * c.d;
  // z.units is a multiple of 8, blockDim.x one of 8: the 4 lanes of a group are always together
  const int step = gridDim.y * blockDim.x;
  for (int u0 = blockIdx.y * blockDim.x; u0 < z.units; u0 += step) {
    const int u = u0 + threadIdx.x;
    const bool in = u < z.units;
    const Unit w = unit_of(in ? u : 0, z.log_chunks);
    const int at = w.h * c.d + w.chunk * 16;
    const T* src = (w.part ? v : k) + at;
    float q[16];                                           // the coordinates, then their codes
    {
      Sixteen<T> raw;
      raw.load(src);
      raw.get(q);
    }
    float lo = q[0], hi = q[0];
#pragma unroll
    for (int i = 1; i < 16; ++i) {
      lo = min_nan(lo, q[i]);
      hi = max_nan(hi, q[i]);
    }
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
      lo = min_nan(lo, __shfl_xor_sync(0xffffffffu, lo, o));
      hi = max_nan(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    }
    // coordinates past the range get the codes of its ends, as the ends themselves would; a NaN makes scale and zero NaN
    // (no quotient is formed then: the codes are 0)
    lo = min_nan(max_nan(lo, -65504.f), 65504.f);
    hi = min_nan(max_nan(hi, -65504.f), 65504.f);
    const __half zh = __float2half_rn(lo + 0.f);           // + 0: a zero has one form
    const float zero = __half2float(zh), span = __fsub_rn(hi, zero);
    const __half sh = __float2half_rn(__fdiv_rn(max_nan(span, 0.f), 15.f));
    const float s = __half2float(sh);
    const float inv = s > 0.f ? __frcp_rn(15.f * s) : 0.f;
    constexpr float kRound = 12582912.f;                   // 1.5 * 2^23
    uint32_t codes[2] = {0, 0};
    float near = 0.f;
#pragma unroll
    for (int i = 15; i >= 0; --i) {
      const float f = __saturatef((q[i] - zero) * inv);
      const float y = fmaf(f, 15.f, kRound);
      q[i] = y - kRound;
      near = fmaxf(near, fabsf(fmaf(f, 15.f, -q[i])));
      codes[i / 8] = (codes[i / 8] << 4) + __float_as_uint(y);
    }
    codes[0] -= 0x3f400000u;                               // 0x4b400000 (1 + 16 + 256 + ...) in 32 bits
    codes[1] -= 0x3f400000u;
    if (near > 0.5f - 1e-5f) {
      float x[16];                                         // read again: this is rare
      Sixteen<T> raw;
      raw.load(src);
      raw.get(x);
      codes[0] = codes[1] = 0;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float f15 = __saturatef((x[i] - zero) * inv) * 15.f, f = floorf(fminf(f15, 14.9f));
        float r = rintf(f15);
        if (fabsf(f15 - f - 0.5f) < 2e-5f) {
          const double border = (static_cast<double>(f) + 0.5) * static_cast<double>(s) + static_cast<double>(zero);
          const double at = static_cast<double>(x[i]);
          r = at > border ? f + 1.f : at < border ? f : 2.f * rintf(0.5f * f + 0.25f);   // a tie: the even one
        }
        q[i] = r;
        codes[i / 8] |= static_cast<uint32_t>(r) << (4 * (i & 7));
      }
    }
    T* values = w.part ? vv : kv;
    if (values && in && live) {
      float val[8];
#pragma unroll
      for (int p = 0; p < 16; p += 8) {
#pragma unroll
        for (int i = 0; i < 8; ++i) val[i] = fmaf(s, q[p + i], zero);
        store8(values + row0 + at + p, val);
      }
    }
    if (stored && in) {
      uint8_t* base = block + w.h * static_cast<int64_t>(z.head_bytes) + w.part * 9 * c.d;
      *reinterpret_cast<uint2*>(base + t * (c.d / 2) + w.chunk * 8) = make_uint2(codes[0], codes[1]);
      if (w.chunk % 4 == 0)
        *reinterpret_cast<uint32_t*>(base + 8 * c.d + t * (c.d / 16) + w.chunk) =
            static_cast<uint32_t>(__half_as_ushort(sh)) | (static_cast<uint32_t>(__half_as_ushort(zh)) << 16);
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) k_kv4_dequant(tq_kv4 c, const int64_t* slots, int64_t n_tokens, T* k, T* v,
                                                          Sizes z) {
  wait_for_stream();
  const int64_t token = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y;
  if (token >= n_tokens) return;
  const int64_t slot = slots[token];
  if (slot < 0) return;
  if (slot >= z.n_slots) {
    if (threadIdx.x == 0 && blockIdx.y == 0 && c.status) atomicOr(c.status, kStatusIndex);
    return;
  }
  int t;
  const uint8_t* block = c.pool + block_of(c, z, slot, t);
  for (int u = blockIdx.y * blockDim.x + threadIdx.x; u < z.units; u += gridDim.y * blockDim.x) {
    const Unit w = unit_of(u, z.log_chunks);
    T* out = w.part ? v : k;
    if (!out) continue;
    const uint8_t* base = block + w.h * static_cast<int64_t>(z.head_bytes) + w.part * 9 * c.d;
    const uint2 codes = *reinterpret_cast<const uint2*>(base + t * (c.d / 2) + w.chunk * 8);
    const uint32_t pair = *reinterpret_cast<const uint32_t*>(base + 8 * c.d + t * (c.d / 16) + (w.chunk / 4) * 4);
    const float s = __half2float(__ushort_as_half(static_cast<unsigned short>(pair & 0xffffu)));
    const float zero = __half2float(__ushort_as_half(static_cast<unsigned short>(pair >> 16)));
    float val[8];
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      const uint32_t word = p ? codes.y : codes.x;
#pragma unroll
      for (int i = 0; i < 8; ++i) val[i] = fmaf(s, static_cast<float>((word >> (4 * i)) & 15u), zero);
      store8(out + token * c.kv_heads * c.d + w.h * c.d + w.chunk * 16 + 8 * p, val);
    }
  }
}

// Threads across a token's units, tokens down.  Many tokens: 64 threads take a
// token, so that its address is worked out once for several units (append of 8
// heads, d = 128, bf16, 64 and 256 threads: 8192 tokens 17.0 and 17.5 us, 16384
// 30.0 and 32.2, 32768 56 and 63); few: a
// thread has one unit, and a token's units may lie in several blocks (up to 4736
// tokens both take the same time).
struct Shape {
  dim3 grid, block;
  Sizes z;
};
Shape shape_of(const tq_kv4& c, int64_t n) {
  Shape s;
  s.z.log_chunks = c.d == 64 ? 2 : c.d == 128 ? 3 : 4;
  s.z.units = c.kv_heads << (s.z.log_chunks + 1);
  s.z.n_slots = c.n_pages * c.page_size;
  s.z.inv_ps = 1.0 / c.page_size;
  s.z.head_bytes = c.page_size / 16 * 18 * c.d;
  s.z.page_bytes = static_cast<uint32_t>(c.kv_heads) * s.z.head_bytes;
  const int most = n >= 148 * 32 ? 64 : kThreads;
  int x = 8;
  while (x < s.z.units && x < most) x <<= 1;
  s.block = dim3(x, kThreads / x);
  const int64_t blocks = (n + s.block.y - 1) / s.block.y;
  const int64_t across = (s.z.units + x - 1) / x, want = (148 * 8 + blocks - 1) / blocks;
  s.grid = dim3(static_cast<unsigned>(blocks), static_cast<unsigned>(across < want ? across : want));
  return s;
}

template <typename T>
int append(const tq_kv4& c, const void* k, int64_t ld_k, const void* v, int64_t ld_v, int64_t n, const int64_t* slots,
           void* kv, void* vv, cudaStream_t st) {
  const Shape s = shape_of(c, n);
  return launch_dependent(k_kv4_append<T>, s.grid, s.block, 0, st, c, static_cast<const T*>(k), ld_k,
                          static_cast<const T*>(v), ld_v, n, slots, static_cast<T*>(kv), static_cast<T*>(vv), s.z);
}

template <typename T>
int dequant(const tq_kv4& c, const int64_t* slots, int64_t n, void* k, void* v, cudaStream_t st) {
  const Shape s = shape_of(c, n);
  return launch_dependent(k_kv4_dequant<T>, s.grid, s.block, 0, st, c, slots, n, static_cast<T*>(k), static_cast<T*>(v), s.z);
}

}  // namespace

int launch_kv4_append(const tq_kv4& c, const void* k, int64_t ld_k, const void* v, int64_t ld_v, int bf16,
                      int64_t n_tokens, const int64_t* slots, void* kv, void* vv, void* stream) {
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return bf16 ? append<__nv_bfloat16>(c, k, ld_k, v, ld_v, n_tokens, slots, kv, vv, st)
              : append<float>(c, k, ld_k, v, ld_v, n_tokens, slots, kv, vv, st);
}

int launch_kv4_dequant(const tq_kv4& c, const int64_t* slots, int64_t n_tokens, void* k, void* v, int bf16,
                       void* stream) {
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return bf16 ? dequant<__nv_bfloat16>(c, slots, n_tokens, k, v, st) : dequant<float>(c, slots, n_tokens, k, v, st);
}

}  // namespace tq
