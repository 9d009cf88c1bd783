// The norms around a block with its gate and residual sum:
//   a = x or norm(x) * post_weight,  h = residual + scale * gate * a,  y = norm(h) * weight.
// One CTA per row; the row stays in registers in fp32 between its two sums, so that every input is
// read once.  Bound by memory: x, residual and gate in, h and y out.  8192 rows of 5120, all in bf16:
// 72 us, 5.8 TB/s.  Rows that no 16-byte load fits (an odd width, stride or offset) go one value at a time, which is bound by
// instructions: 8192 rows of 5119 222 us, of 2001 63; above 8192 wide the 16 values a thread holds of x, residual and gate
// spill (184 bytes): 4096 rows of 16383 479 us.
#include <cuda_bf16.h>

#include "actq.cuh"
#include "common.cuh"
#include "kernels.h"

namespace vt {

namespace {

// V values of a row as they lie (V = 8: 16-byte loads; V = 1: any alignment and stride), bf16 or
// either type.
template <int V>
struct Raw {
  uint32_t w[V == 8 ? 4 : 1];
};
template <int V>
struct RawAny {
  uint32_t w[V];
};
template <int V>
__device__ __forceinline__ void fetch(Raw<V>& r, const void* base, int64_t at) {
  const __nv_bfloat16* p = reinterpret_cast<const __nv_bfloat16*>(base) + at;
  if constexpr (V == 8) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    r.w[0] = v.x, r.w[1] = v.y, r.w[2] = v.z, r.w[3] = v.w;
  } else {
    r.w[0] = *reinterpret_cast<const uint16_t*>(p);
  }
}
template <int V>
__device__ __forceinline__ void widen(const Raw<V>& r, float (&x)[V]) {
  if constexpr (V == 8) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      x[2 * q] = bf16_lo(r.w[q]);
      x[2 * q + 1] = bf16_hi(r.w[q]);
    }
  } else {
    x[0] = bf16_lo(r.w[0]);
  }
}
template <int V>
__device__ __forceinline__ void fetch_any(RawAny<V>& r, const void* base, int fp32, int64_t at) {
  if (fp32) {
    const float* p = reinterpret_cast<const float*>(base) + at;
    if constexpr (V == 8) {
      const uint4 a = reinterpret_cast<const uint4*>(p)[0], b = reinterpret_cast<const uint4*>(p)[1];
      r.w[0] = a.x, r.w[1] = a.y, r.w[2] = a.z, r.w[3] = a.w, r.w[4] = b.x, r.w[5] = b.y, r.w[6] = b.z, r.w[7] = b.w;
    } else {
      r.w[0] = *reinterpret_cast<const uint32_t*>(p);
    }
  } else {
    Raw<V> h;
    fetch(h, base, at);
#pragma unroll
    for (int i = 0; i < (V == 8 ? 4 : 1); ++i) r.w[i] = h.w[i];
  }
}
template <int V>
__device__ __forceinline__ void widen_any(const RawAny<V>& r, int fp32, float (&x)[V]) {
  if (fp32) {
#pragma unroll
    for (int i = 0; i < V; ++i) x[i] = __uint_as_float(r.w[i]);
  } else {
    Raw<V> h;
#pragma unroll
    for (int i = 0; i < (V == 8 ? 4 : 1); ++i) h.w[i] = r.w[i];
    widen(h, x);
  }
}
template <int V>
__device__ __forceinline__ void load_any(const void* base, int fp32, int64_t at, float (&x)[V]) {
  RawAny<V> r;
  fetch_any(r, base, fp32, at);
  widen_any(r, fp32, x);
}
template <int V>
__device__ __forceinline__ void store_any(void* base, int fp32, int64_t at, const float (&x)[V]) {
  if (fp32) {
    float* p = reinterpret_cast<float*>(base) + at;
    if constexpr (V == 8) {
      reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
      reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
    } else {
      *p = x[0];
    }
    return;
  }
  __nv_bfloat16* p = reinterpret_cast<__nv_bfloat16*>(base) + at;
  if constexpr (V == 8) {
    uint32_t w[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * q], x[2 * q + 1]);
      w[q] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
    *p = __float2bfloat16(x[0]);
  }
}

// Sum over the CTA, the same value (and the same order of additions) in every thread.
__device__ __forceinline__ float block_sum(float v, float* red, int warps) {
#pragma unroll
  for (int m = 16; m; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
  if (warps == 1) return v;
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  float t = (threadIdx.x & 31) < warps ? red[threadIdx.x & 31] : 0.0f;
#pragma unroll
  for (int m = 16; m; m >>= 1) t += __shfl_xor_sync(0xffffffffu, t, m);
  return t;
}

// N chunks of V values per thread: element (i * blockDim + tid) * V.
template <int V, int N>
__global__ void __launch_bounds__(1024) k_norm(const NormLaunch p) {
  __shared__ float red[2][32];
  const int64_t t = blockIdx.x;
  const int H = (int)p.H, warps = blockDim.x >> 5;
  // everything that the row needs is under way before the first sum
  Raw<V> x[N], gate[N];
  RawAny<V> res[N];
  float a[N][V];
  float ss = 0.0f;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int e = (i * blockDim.x + threadIdx.x) * V;
    if (e < H) {
      fetch(x[i], p.x, t * p.ldx + e);
      if (p.gate) fetch(gate[i], p.gate, t * p.ldg + e);
      if (p.residual) fetch_any(res[i], p.residual, p.residual_fp32, t * p.ldr + e);
    }
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int e = (i * blockDim.x + threadIdx.x) * V;
    if (e < H) {
      widen(x[i], a[i]);
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j) a[i][j] = 0.0f;
    }
  }
  if (p.post_weight) {
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int j = 0; j < V; ++j) ss += a[i][j] * a[i][j];
    const float r = 1.0f / sqrtf(block_sum(ss, red[0], warps) / (float)H + p.eps);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int e = (i * blockDim.x + threadIdx.x) * V;
      if (e < H) {
        float w[V];
        load_any<V>(p.post_weight, p.weights_fp32, e, w);
#pragma unroll
        for (int j = 0; j < V; ++j) a[i][j] *= r * w[j];
      }
    }
  }
  ss = 0.0f;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int e = (i * blockDim.x + threadIdx.x) * V;
    if (e < H) {
      if (p.gate) {
        float g[V];
        widen(gate[i], g);
#pragma unroll
        for (int j = 0; j < V; ++j) a[i][j] *= g[j];
      }
#pragma unroll
      for (int j = 0; j < V; ++j) a[i][j] *= p.scale;
      if (p.residual) {
        float r[V];
        widen_any(res[i], p.residual_fp32, r);
#pragma unroll
        for (int j = 0; j < V; ++j) a[i][j] += r[j];
        store_any<V>(p.h, p.residual_fp32, t * p.ldh + e, a[i]);
      }
#pragma unroll
      for (int j = 0; j < V; ++j) ss += a[i][j] * a[i][j];
    }
  }
  const float r = 1.0f / sqrtf(block_sum(ss, red[1], warps) / (float)H + p.eps);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int e = (i * blockDim.x + threadIdx.x) * V;
    if (e < H) {
      float w[V];
      load_any<V>(p.weight, p.weights_fp32, e, w);
#pragma unroll
      for (int j = 0; j < V; ++j) a[i][j] *= r * w[j];
      store_any<V>(p.y, 0, t * p.ldy + e, a[i]);
    }
  }
}

constexpr int kOne = 256;

inline bool on16(const void* p) { return ((uintptr_t)p & 15) == 0; }

}  // namespace

cudaError_t launch_norm(const NormLaunch& L, cudaStream_t s) {
  const int64_t rm = L.residual_fp32 ? 3 : 7;  // a row's stride in elements: 16 bytes at least
  const bool vec = L.H % 8 == 0 && on16(L.x) && L.ldx % 8 == 0 && on16(L.y) && L.ldy % 8 == 0 &&
                   on16(L.weight) && on16(L.post_weight) && on16(L.gate) && L.ldg % 8 == 0 &&
                   on16(L.residual) && on16(L.h) && (L.ldr & rm) == 0 && (L.ldh & rm) == 0;
  const int64_t chunks = vec ? L.H / 8 : L.H;
  // one vector a thread up to rows of 2048, two above (us, one and two: 203 rows of 2048 3.0 and 3.5, 8192 of 2048 34 and 29,
  // 8192 of 4096 77 and 56); one value at a time, 8 a thread as long as 1024 threads are enough (8, 2 and 4 of them: 8192 rows
  // of 1001 29, 43 and 33, of 2001 63, 95 and 65; 1 row of 2001 4.0, 3.6 and 3.4; 16 take 222 to 286 at 5119)
  const int n = vec ? (chunks <= kOne ? 1 : 2) : (chunks <= 8192 ? 8 : 16);
  const int threads = (int)(((chunks + n - 1) / n + 31) / 32 * 32);
  const unsigned rows = (unsigned)L.T;
  if (vec) {
    if (n == 1) k_norm<8, 1><<<rows, threads, 0, s>>>(L);
    else k_norm<8, 2><<<rows, threads, 0, s>>>(L);
  } else {
    if (n == 8) k_norm<1, 8><<<rows, threads, 0, s>>>(L);
    else k_norm<1, 16><<<rows, threads, 0, s>>>(L);
  }
  return cudaGetLastError();
}

}  // namespace vt
