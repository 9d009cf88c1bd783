// Low-rank adapters of many requests beside a shared projection:
//   out[m] = y[m] + scale[a] * B_a (A_a x[m]),  a the adapter of row m's group.
#include <cuda_bf16.h>

#include "common.cuh"
#include "kernels.h"

namespace vt {

namespace {

// One block per grouped row: v = A_a x (one warp per rank), then out = y + scale * B_a v.
__global__ void __launch_bounds__(256) k_lora_simple(const LoraLaunch L) {
  __shared__ float s_v[kMaxRank];
  __shared__ int s_e;
  const int64_t i = blockIdx.x;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t m = L.order[i];
  if (m < 0 || m >= L.M) return;
  if (threadIdx.x == 0) {
    s_e = -1;
    for (int e = 0; e < L.L; ++e)
      if (L.offsets[e] <= i && i < L.offsets[e + 1]) s_e = e;
  }
  __syncthreads();
  const int e = s_e;
  int R = e < 0 ? 0 : L.R;
  if (e >= 0 && L.ranks) R = L.ranks[e] < 0 ? 0 : (L.ranks[e] < L.R ? L.ranks[e] : L.R);
  const __nv_bfloat16* x = reinterpret_cast<const __nv_bfloat16*>(L.x) + m * L.ldx;
  for (int r = warp; r < R; r += 8) {
    const __nv_bfloat16* a = reinterpret_cast<const __nv_bfloat16*>(L.A) + ((int64_t)e * L.R + r) * L.K;
    float v = 0.0f;
    for (int64_t k = lane; k < L.K; k += 32) v += __bfloat162float(a[k]) * __bfloat162float(x[k]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (lane == 0) s_v[r] = v * L.scale[e];
  }
  __syncthreads();
  const __nv_bfloat16* y = reinterpret_cast<const __nv_bfloat16*>(L.y) + m * L.ldy;
  __nv_bfloat16* out = reinterpret_cast<__nv_bfloat16*>(L.out) + m * L.ldo;
  for (int64_t n = threadIdx.x; n < L.N; n += 256) {
    float v = 0.0f;
    if (R) {
      const __nv_bfloat16* b = reinterpret_cast<const __nv_bfloat16*>(L.B) + ((int64_t)e * L.N + n) * L.R;
      for (int r = 0; r < R; ++r) v += __bfloat162float(b[r]) * s_v[r];
    }
    out[n] = __float2bfloat16_rn(__bfloat162float(y[n]) + v);
  }
}

}  // namespace

cudaError_t launch_lora(const LoraLaunch& L, cudaStream_t s) {
  k_lora_simple<<<(unsigned)L.M, 256, 0, s>>>(L);
  return cudaGetLastError();
}

}  // namespace vt
