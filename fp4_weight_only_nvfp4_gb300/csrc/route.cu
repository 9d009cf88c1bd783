// Router and grouping of rows by an index: the top-k experts of each token by a total order,
// their weights, and the (token, slot) pairs in stable index order.  Source for the order:
// "re-verify 27B NVFP4 on the nvidia ModelOpt checkpoint" (vllm.cpp PR #178), "Speed --
// warp-shuffle MoE router top-k" (any reduction order gives the same (value, index)).
#include <cuda_bf16.h>

#include "common.cuh"
#include "kernels.h"

namespace vt {

namespace {

// Scores as integers whose order is the scores' total order: larger score, larger key; -0
// equals +0; NaN above every number; -inf (a masked expert) is 0, the key of "no candidate".
__device__ __forceinline__ uint32_t score_key(float v) {
  if (v != v) return 0xFFFFFFFFu;
  const uint32_t b = v == 0.0f ? 0u : __float_as_uint(v);
  const uint32_t k = (b & 0x80000000u) ? ~b : (b | 0x80000000u);
  return k == 0x007FFFFFu ? 0u : k;  // ~bits(-inf)
}

__device__ __forceinline__ float load_logit(const void* p, int bf16, int64_t i) {
  return bf16 ? __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(p)[i])
              : reinterpret_cast<const float*>(p)[i];
}

constexpr int kRouteWarps = 8;
constexpr int kPerLane = kMaxGroups / 32;

// One warp per token: every lane keeps its E / 32 keys in registers; topk times the warp takes
// the largest key (lowest index among equals) and removes it.
__global__ void __launch_bounds__(kRouteWarps * 32) k_topk(const RouteLaunch L) {
  const int lane = threadIdx.x & 31;
  const int64_t m = (int64_t)blockIdx.x * kRouteWarps + (threadIdx.x >> 5);
  if (m >= L.M) return;
  uint32_t key[kPerLane];
  float mx = -INFINITY, sum = 0.0f;
#pragma unroll
  for (int i = 0; i < kPerLane; ++i) {
    const int e = i * 32 + lane;
    key[i] = 0;
    if (e < L.E) {
      const float l = load_logit(L.logits, L.bf16, m * L.ld + e);
      float sc = l;
      if (L.scoring == 1) {
        sc = 1.0f / (1.0f + expf(-l));
        if (L.bias) sc += L.bias[e];
      }
      key[i] = l == -INFINITY ? 0u : score_key(sc);
      mx = fmaxf(mx, l);
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  if (L.scoring == 0) {
#pragma unroll
    for (int i = 0; i < kPerLane; ++i) {
      const int e = i * 32 + lane;
      if (e < L.E && key[i]) sum += expf(load_logit(L.logits, L.bf16, m * L.ld + e) - mx);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  }
  int id = -1;        // lane j: the j-th choice
  float w = 0.0f;
  for (int j = 0; j < L.topk; ++j) {
    uint32_t best = 0;
    int at = 0x7FFFFFFF;
#pragma unroll
    for (int i = 0; i < kPerLane; ++i)
      if (key[i] > best) {
        best = key[i];
        at = i * 32 + lane;
      }
    const uint32_t top = __reduce_max_sync(0xffffffffu, best);
    if (top == 0) break;
    const int e = __reduce_min_sync(0xffffffffu, best == top ? at : 0x7FFFFFFF);
#pragma unroll
    for (int i = 0; i < kPerLane; ++i)
      if (i * 32 + lane == e) key[i] = 0;
    if (lane == j) {
      id = e;
      const float l = load_logit(L.logits, L.bf16, m * L.ld + e);
      w = L.scoring == 1 ? 1.0f / (1.0f + expf(-l)) : expf(l - mx) / sum;
    }
  }
  if (L.renormalize) {
    float s = w;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (id >= 0) w /= s;
  }
  if (lane < L.topk) {
    L.ids[m * L.topk + lane] = id;
    L.weights[m * L.topk + lane] = id >= 0 ? w * L.scale : 0.0f;
  }
}

// Group e's pairs (block e; block E: the pairs in no group): counted, then, once every count
// is known, written in pair order.
constexpr int kGroupBlock = 256;
__device__ __forceinline__ bool in_group(int id, int e, int E) {
  return e < E ? id == e : (id < 0 || id >= E);
}

__global__ void __launch_bounds__(kGroupBlock) k_count(const int32_t* ids, int64_t P, int E,
                                                       int* counts) {
  __shared__ int total;
  if (threadIdx.x == 0) total = 0;
  __syncthreads();
  int n = 0;
  for (int64_t i = threadIdx.x; i < P; i += kGroupBlock) n += in_group(ids[i], blockIdx.x, E);
  atomicAdd(&total, n);
  __syncthreads();
  if (threadIdx.x == 0) counts[blockIdx.x] = total;
}

__global__ void __launch_bounds__(kGroupBlock) k_scatter(const int32_t* ids, int64_t P, int E,
                                                         const int* counts, int32_t* order,
                                                         int32_t* offsets) {
  __shared__ int s_base, s_warp[kGroupBlock / 32];
  const int e = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    int b = 0;
    for (int i = 0; i < e; ++i) b += counts[i];
    s_base = b;
    offsets[e] = b;  // block E: the number of grouped pairs
  }
  __syncthreads();
  int base = s_base;
  for (int64_t i0 = 0; i0 < P; i0 += kGroupBlock) {
    const int64_t i = i0 + threadIdx.x;
    const bool in = i < P && in_group(ids[i], e, E);
    const uint32_t b = __ballot_sync(0xffffffffu, in);
    if (lane == 0) s_warp[warp] = __popc(b);
    __syncthreads();
    int before = __popc(b & ((1u << lane) - 1u)), all = 0;
    for (int w = 0; w < kGroupBlock / 32; ++w) {
      if (w < warp) before += s_warp[w];
      all += s_warp[w];
    }
    if (in) order[base + before] = (int32_t)i;
    base += all;
    __syncthreads();
  }
}

}  // namespace

size_t route_workspace_bytes(int64_t pairs, int64_t E) {
  (void)pairs;
  return 256 + ((size_t)(E + 1) * 4 + 255) / 256 * 256;
}

cudaError_t launch_route(const RouteLaunch& L, cudaStream_t s) {
  int* counts = reinterpret_cast<int*>(reinterpret_cast<uint8_t*>(L.workspace) + 256);
  const int64_t P = L.M * L.topk;
  if (L.logits && L.M)
    k_topk<<<(unsigned)((L.M + kRouteWarps - 1) / kRouteWarps), kRouteWarps * 32, 0, s>>>(L);
  k_count<<<L.E + 1, kGroupBlock, 0, s>>>(L.ids, P, L.E, counts);
  k_scatter<<<L.E + 1, kGroupBlock, 0, s>>>(L.ids, P, L.E, counts, L.order, L.offsets);
  return cudaGetLastError();
}

}  // namespace vt
