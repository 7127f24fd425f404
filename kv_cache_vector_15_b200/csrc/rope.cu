// RMS norm of each head of q and k and the rotary rotation, in one pass.
//
// Bound: the bytes of q and k, read and written once (2 d esz per row).  One
// block takes a token (or, for few tokens, a part of its heads): the angles of
// a token are shared by its heads, so they are formed once per block, in fp64
// (position * inv_freq in turns, reduced by rint before the conversion to
// fp32: an fp32 product would lose all of the fraction at positions near
// 2^24), and kept in shared memory with the norm's weights multiplied in: a
// pair's four factors are one 16-byte read per row.  A row is held by d / 8
// lanes, each with four whole pairs of the rotation: (i, i + rot / 2) are two
// 8- or 16-byte loads 4 coordinates wide, so neither the rotation nor the
// store needs data of another lane; only the sum of squares is exchanged
// (3 to 5 shuffles).  Half-split rotations whose rot / 2 is no multiple of 4
// take one pair per lane and step (their loads cannot be wider).  Three rows of
// a lane are loaded before the angles are formed.  8192 tokens of 32 + 8 heads,
// d = 128, bf16 (168 MB): 36 to 37 us, 4.6 TB/s; a row's address worked out from the
// kernel's arguments 38 us; one row ahead 51 us; with the cosines and the weights
// apart and bank conflicts 61 us.  Issue slots are taken in 69 % of the cycles, and
// between warps wait at the block's barrier for the angles, and for shared memory;
// the next token's rows
// loaded under this one's (4 tokens a block) cost registers and occupancy: 43 us;
// 4 blocks an SM instead of 5 39 us, 6 (spills) 38 us.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "kv4_internal.h"
#include "launch.cuh"
#include "tq_internal.h"

namespace tq {
namespace {

constexpr int kThreads = 256;

// Four neighbouring coordinates as they were loaded, and as numbers.
template <typename T>
struct Four;
template <>
struct Four<float> {
  float4 t;
  __device__ __forceinline__ void load(const float* p) { t = *reinterpret_cast<const float4*>(p); }
  __device__ __forceinline__ void get(float (&v)[4]) const { v[0] = t.x; v[1] = t.y; v[2] = t.z; v[3] = t.w; }
};
template <>
struct Four<__nv_bfloat16> {
  uint2 t;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { t = *reinterpret_cast<const uint2*>(p); }
  __device__ __forceinline__ void get(float (&v)[4]) const {
    v[0] = __uint_as_float(t.x << 16); v[1] = __uint_as_float(t.x & 0xffff0000u);
    v[2] = __uint_as_float(t.y << 16); v[3] = __uint_as_float(t.y & 0xffff0000u);
  }
};
template <typename T>
__device__ __forceinline__ void store4(T* p, const float (&v)[4]);
template <>
__device__ __forceinline__ void store4<float>(float* p, const float (&v)[4]) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
}
template <>
__device__ __forceinline__ void store4<__nv_bfloat16>(__nv_bfloat16* p, const float (&v)[4]) {
  __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), b = __floats2bfloat162_rn(v[2], v[3]);
  uint2 t;
  t.x = *reinterpret_cast<uint32_t*>(&a);
  t.y = *reinterpret_cast<uint32_t*>(&b);
  *reinterpret_cast<uint2*>(p) = t;
}
__device__ __forceinline__ float load1(const float* p) { return *p; }
__device__ __forceinline__ float load1(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void store1(float* p, float v) { *p = v; }
__device__ __forceinline__ void store1(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// V pairs per lane and step: 4, or 1 where the pairs' halves cannot be loaded four wide.
template <typename T, int D, int V, bool kInter>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 ? 5 : 4) k_qk_norm_rope(const __grid_constant__ RopeArgs a) {
  constexpr int kLanes = V == 4 ? D / 8 : 32;             // lanes per row
  constexpr int kSteps = D / 2 / (kLanes * V);            // steps of V pairs per lane
  constexpr int kGroups = kThreads / kLanes;
  constexpr int kRows = 3;                                // rows of a lane in flight at a time
  static_assert(V == 1 || kSteps == 1, "a lane has its four pairs in one step");
  // per matrix and pair: w0 cos, w1 sin, w0 sin, w1 cos (past the rotated pairs cos = 1, sin = 0); pair p stands at
  // place_of(p), so that lanes reading their j-th pairs read neighbouring places
  __shared__ float4 factors[2][D / 2];
  auto place_of = [](int p) { return p % V * (D / 2 / V) + p / V; };
  wait_for_stream();
  const int64_t token = blockIdx.x;
  const int n_pairs = a.rot_dim / 2, heads = a.heads[0] + a.heads[1];
  const int lane = threadIdx.x % kLanes, group = threadIdx.x / kLanes;
  const int stride = gridDim.y * kGroups;

  // pair p of a row stands at coordinates (at0, at1)
  auto at0 = [&](int p) { return kInter ? 2 * p : p < n_pairs ? p : a.rot_dim + (p - n_pairs) / V * 2 * V + (p - n_pairs) % V; };
  auto at1 = [&](int p) { return kInter ? 2 * p + 1 : p < n_pairs ? p + n_pairs : at0(p) + V; };
  // where a lane's first pair stands in row 0 of each matrix, the rows of k counted on from those of q: a row's
  // address is one multiplication and one choice
  const int of0 = at0(lane * V), of1 = kInter ? of0 + V : at1(lane * V);
  const T* const xq = static_cast<const T*>(a.x[0]) + token * a.ld_x[0] + of0;
  const T* const xk = static_cast<const T*>(a.x[1]) + token * a.ld_x[1] - static_cast<int64_t>(a.heads[0]) * D + of0;
  T* const yq = static_cast<T*>(a.y[0]) + token * a.ld_y[0] + of0;
  T* const yk = static_cast<T*>(a.y[1]) + token * a.ld_y[1] - static_cast<int64_t>(a.heads[0]) * D + of0;
  const int apart = of1 - of0;
  // a lane's part of kRows rows as they were loaded
  Four<T> raw[kRows][V == 4 ? 2 : 1];
  float ones[V == 4 ? 1 : kRows][kSteps][2];
  auto fetch = [&](int row, int k) {
    const T* x = (row >= a.heads[0] ? xk : xq) + static_cast<int64_t>(row) * D;
    if constexpr (V == 4) {
      raw[k][0].load(x);
      raw[k][1].load(x + apart);
    } else {
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        ones[k][s][0] = load1(x - of0 + at0(s * kLanes + lane));
        ones[k][s][1] = load1(x - of0 + at1(s * kLanes + lane));
      }
    }
  };
  auto numbers = [&](int k, float (&u)[kSteps][V], float (&v)[kSteps][V]) {
    if constexpr (V == 4) {
      float t0[4], t1[4];
      raw[k][0].get(t0);
      raw[k][1].get(t1);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        u[0][j] = !kInter ? t0[j] : j < 2 ? t0[2 * (j & 1)] : t1[2 * (j & 1)];
        v[0][j] = !kInter ? t1[j] : j < 2 ? t0[2 * (j & 1) + 1] : t1[2 * (j & 1) + 1];
      }
    } else {
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        u[s][0] = ones[k][s][0];
        v[s][0] = ones[k][s][1];
      }
    }
  };

  const int row0 = blockIdx.y * kGroups + group;
#pragma unroll
  for (int k = 0; k < kRows; ++k)
    if (row0 + k * stride < heads) fetch(row0 + k * stride, k);      // in flight while the angles are formed
  for (int i = threadIdx.x; i < D / 2; i += kThreads) {
    float c = 1.f, s = 0.f;
    if (i < n_pairs) {
      double t = static_cast<double>(a.positions[a.axis[i] * a.n_tokens + token]) * a.turns[i];
      t -= rint(t);
      sincospif(static_cast<float>(2.0 * t), &s, &c);
    }
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      const float* w = a.w[m];
      const float w0 = w ? __ldg(w + at0(i)) : 1.f, w1 = w ? __ldg(w + at1(i)) : 1.f;
      factors[m][place_of(i)] = make_float4(w0 * c, w1 * s, w0 * s, w1 * c);
    }
  }
  __syncthreads();

  // whole warps stay in the loop together: the shuffles below need them
  for (int base = blockIdx.y * kGroups; base < heads; base += kRows * stride) {
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
      if (base + k * stride >= heads) break;   // the same for the whole block
      const int row = base + group + k * stride;
      float u[kSteps][V], v[kSteps][V], sum = 0.f;
      numbers(k, u, v);
#pragma unroll
      for (int s = 0; s < kSteps; ++s)
#pragma unroll
        for (int j = 0; j < V; ++j) sum = fmaf(u[s][j], u[s][j], fmaf(v[s][j], v[s][j], sum));
#pragma unroll
      for (int o = kLanes / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      if (row < heads) {
        const float r = rsqrtf(sum * (1.f / D) + a.eps);
        const int which = row >= a.heads[0];
        const float4* f = factors[which];
        T* y = (which ? yk : yq) + static_cast<int64_t>(row) * D;
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
          const int p = (s * kLanes + lane) * V;
          float nu[V], nv[V];
#pragma unroll
          for (int j = 0; j < V; ++j) {
            const float4 e = f[place_of(p + j)];
            const float x0 = u[s][j] * r, x1 = v[s][j] * r;
            nu[j] = fmaf(x0, e.x, -(x1 * e.y));
            nv[j] = fmaf(x0, e.z, x1 * e.w);
          }
          if constexpr (V == 4 && kInter) {
            const float t0[4] = {nu[0], nv[0], nu[1], nv[1]}, t1[4] = {nu[2], nv[2], nu[3], nv[3]};
            store4(y, t0);
            store4(y + apart, t1);
          } else if constexpr (V == 4) {
            store4(y, nu);
            store4(y + apart, nv);
          } else {
            store1(y - of0 + at0(p), nu[0]);
            store1(y - of0 + at1(p), nv[0]);
          }
        }
      }
    }
#pragma unroll
    for (int k = 0; k < kRows; ++k) {          // more than kRows rows a lane: the next ones
      const int row = base + group + (kRows + k) * stride;
      if (row < heads) fetch(row, k);
    }
  }
}

template <typename T, int D, int V, bool kInter>
int launch(const RopeArgs& a, cudaStream_t st) {
  constexpr int kGroups = kThreads / (V == 4 ? D / 8 : 32);
  const int heads = a.heads[0] + a.heads[1];
  // few tokens: a token's heads over several blocks, up to two blocks per SM
  const int64_t most = (heads + kGroups - 1) / kGroups, want = (296 + a.n_tokens - 1) / a.n_tokens;
  const dim3 grid(static_cast<unsigned>(a.n_tokens), static_cast<unsigned>(most < want ? most : want));
  return launch_dependent(k_qk_norm_rope<T, D, V, kInter>, grid, dim3(kThreads), 0, st, a);
}

template <typename T, int D>
int launch_d(const RopeArgs& a, cudaStream_t st) {
  if (a.interleaved) return launch<T, D, 4, true>(a, st);
  return a.rot_dim % 8 == 0 ? launch<T, D, 4, false>(a, st) : launch<T, D, 1, false>(a, st);
}

template <typename T>
int launch_t(const RopeArgs& a, cudaStream_t st) {
  if (a.d == 64) return launch_d<T, 64>(a, st);
  return a.d == 128 ? launch_d<T, 128>(a, st) : launch_d<T, 256>(a, st);
}

}  // namespace

int launch_qk_norm_rope(const RopeArgs& a, int bf16, void* stream) {
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return bf16 ? launch_t<__nv_bfloat16>(a, st) : launch_t<float>(a, st);
}

}  // namespace tq
