// Products of ragged groups of rows: C[i] = A[row(i)] . W_e^T for the rows of every expert e in
// one call, with the packed FP4 weights dequantised inside.  Source: "dense projections take
// vLLM's own dense marlin" (vllm.cpp PR #54: the multi-expert route of the same W4A16 GEMM).
#include <cuda_bf16.h>

#include "common.cuh"
#include "kernels.h"

namespace vt {

namespace {

constexpr int kRows = 16;      // grouped rows per tile
constexpr int kThreads = 256;

__device__ __forceinline__ float silu_f(float x) { return x / (1.0f + expf(-x)); }

__device__ __forceinline__ float code_value(uint32_t c) {
  const float m = (c & 6) ? __uint_as_float(((((c >> 1) & 3u) + 126u) << 23) | ((c & 1u) << 22))
                          : 0.5f * (float)(c & 1);
  return (c & 8) ? -m : m;
}

// Offsets are device data of the caller's: one that is out of range must not become an address.
__device__ __forceinline__ int64_t offset_at(const int32_t* offsets, int e, int64_t P) {
  const int64_t v = offsets[e];
  return v < 0 ? 0 : (v > P ? P : v);
}

// One block: 128 packed rows of one expert x 16 of its rows; 256 threads, each one packed row
// and 8 of the 16 rows.
__global__ void __launch_bounds__(kThreads) k_ragged_simple(const RaggedLaunch L) {
  __shared__ float s_a[kRows][kTileK + 1];
  __shared__ uint8_t s_w[kTileBytesNV];
  __shared__ float s_u[kRows][64 + 1];
  __shared__ int64_t s_i0;
  __shared__ int s_n, s_e;
  if (threadIdx.x == 0) {
    int64_t left = blockIdx.y;
    s_n = 0;
    for (int e = 0; e < L.E; ++e) {
      const int64_t b = offset_at(L.offsets, e, L.pairs), n = offset_at(L.offsets, e + 1, L.pairs) - b;
      if (n <= 0) continue;
      const int64_t t = (n + kRows - 1) / kRows;
      if (left < t) {
        s_e = e;
        s_i0 = b + left * kRows;
        s_n = (int)(n - left * kRows < kRows ? n - left * kRows : kRows);
        break;
      }
      left -= t;
    }
  }
  __syncthreads();
  const int n = s_n;
  if (n == 0) return;
  const int64_t i0 = s_i0, rt = blockIdx.x;
  const uint8_t* packed = reinterpret_cast<const uint8_t*>(L.packed) + s_e * L.expert_bytes;
  const PackedHeader* hdr = reinterpret_cast<const PackedHeader*>(packed);
  const int TB = tile_bytes(L.fmt);
  const bool wide = L.fmt == FMT_MX && hdr->wide;
  const int r = threadIdx.x & 127, half = threadIdx.x >> 7;
  const int j = r >> 4, g = r & 7, h = (r >> 3) & 1;
  const __nv_bfloat16* A = reinterpret_cast<const __nv_bfloat16*>(L.A);
  float acc[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  for (int64_t kt = 0; kt < L.KT; ++kt) {
    __syncthreads();
    const uint8_t* src = packed + kHeaderBytes + (rt * L.KT + kt) * TB;
    for (int i = threadIdx.x; i < TB / 16; i += kThreads)
      reinterpret_cast<uint4*>(s_w)[i] = reinterpret_cast<const uint4*>(src)[i];
    for (int i = threadIdx.x; i < kRows * kTileK; i += kThreads) {
      const int row = i / kTileK;
      const int64_t k = kt * kTileK + i % kTileK;
      float v = 0.0f;
      if (row < n && k < L.K) {
        int64_t ar = i0 + row;
        if (L.gather) {
          const int64_t p = L.order[i0 + row];
          ar = p >= 0 && p < L.pairs ? p / L.topk : -1;
        }
        if (ar >= 0) v = __bfloat162float(A[ar * L.lda + k]);
      }
      s_a[row][i % kTileK] = v;
    }
    __syncthreads();
    for (int t = 0; t < 4; ++t) {
      const uint32_t sb = s_w[scale_offset(L.fmt, j, g, t) + h];
      float sc;
      if (L.fmt == FMT_NV) {
        const uint32_t f = e4m3x2_to_f16x2(sb);
        sc = __low2float(*reinterpret_cast<const __half2*>(&f));
      } else if (wide) {
        sc = e8m0_to_f32(sb);
      } else {
        const uint32_t f = mxenc2_to_f16x2(sb);
        sc = __low2float(*reinterpret_cast<const __half2*>(&f));
      }
      for (int q = 0; q < 4; ++q) {
        for (int kk = 0; kk < 4; ++kk) {
          const uint32_t byte = s_w[j * 512 + (4 * g + t) * 16 + 4 * q + (kk & 2) + h];
          const float w = code_value((kk & 1) ? byte >> 4 : byte & 15u) * sc;
#pragma unroll
          for (int m = 0; m < 8; ++m) acc[m] += s_a[half * 8 + m][16 * t + 4 * q + kk] * w;
        }
      }
    }
  }
  __nv_bfloat16* C = reinterpret_cast<__nv_bfloat16*>(L.C);
  const int64_t row = packed_to_row(L.layout, rt * kTileRows + r, L.N, L.seg_split);
  const float f = hdr->factor[row >= L.seg_split ? 1 : 0];
  if (L.silu) {
    __syncthreads();
    if (r >= 64)
      for (int m = 0; m < 8; ++m) s_u[half * 8 + m][r - 64] = acc[m] * f;
    __syncthreads();
  }
  if (row < 0 || (L.silu && r >= 64)) return;
  for (int m = 0; m < 8; ++m) {
    const int i = half * 8 + m;
    if (i >= n) break;
    int64_t cr = i0 + i;
    if (L.scatter) {
      cr = L.order[i0 + i];
      if (cr < 0 || cr >= L.pairs) continue;
    }
    float v = acc[m] * f;
    if (L.silu) v = silu_f(v) * s_u[i][r];
    C[cr * L.ldc + row] = __float2bfloat16_rn(v);
  }
}

// Weighted sum of each token's pairs, in slot order, in fp32.
__global__ void __launch_bounds__(256) k_combine(const __nv_bfloat16* D, int64_t M, int topk,
                                                 int64_t N, int64_t ldd, const int32_t* ids, int E,
                                                 const float* weights, __nv_bfloat16* out,
                                                 int64_t ldo) {
  const int64_t m = blockIdx.y, n = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (n >= N) return;
  float acc = 0.0f;
  for (int j = 0; j < topk; ++j) {
    const int64_t p = m * topk + j;
    if (ids[p] >= 0 && ids[p] < E) acc += weights[p] * __bfloat162float(D[p * ldd + n]);
  }
  out[m * ldo + n] = __float2bfloat16_rn(acc);
}

}  // namespace

cudaError_t launch_ragged(const RaggedLaunch& L, cudaStream_t s) {
  // tiles of 16 rows: at most one partial tile per group in use
  const int64_t groups = L.pairs < L.E ? L.pairs : L.E;
  const int64_t tiles = groups + L.pairs / kRows;
  k_ragged_simple<<<dim3((unsigned)L.RT, (unsigned)(tiles < 65535 ? tiles : 65535)), kThreads, 0, s>>>(L);
  return cudaGetLastError();
}

cudaError_t launch_combine(const void* D, int64_t M, int topk, int64_t N, int64_t ldd,
                           const int32_t* ids, int E, const float* weights, void* out,
                           int64_t ldo, cudaStream_t s) {
  k_combine<<<dim3((unsigned)((N + 255) / 256), (unsigned)M), 256, 0, s>>>(
      reinterpret_cast<const __nv_bfloat16*>(D), M, topk, N, ldd, ids, E, weights,
      reinterpret_cast<__nv_bfloat16*>(out), ldo);
  return cudaGetLastError();
}

}  // namespace vt
