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

// Sorts a lane's PER keys, largest first, equal ones in their order; at[i]: 32 times the i-th's
// place before.
template <int PER>
__device__ __forceinline__ void sort_keys(uint32_t (&key)[PER], uint32_t (&at)[PER]) {
#pragma unroll
  for (int i = 0; i < PER; ++i) at[i] = i * 32;
  // odd-even transposition: neighbours only, so equal keys never pass one another
#pragma unroll
  for (int r = 0; r < PER; ++r)
#pragma unroll
    for (int i = r & 1; i + 1 < PER; i += 2) {
      const bool swap = key[i] < key[i + 1];
      const uint32_t k = key[i], a = at[i];
      key[i] = swap ? key[i + 1] : k;
      key[i + 1] = swap ? k : key[i + 1];
      at[i] = swap ? at[i + 1] : a;
      at[i + 1] = swap ? a : at[i + 1];
    }
}

// One token per warp: lane j of the first topk returns its j-th choice and weight (id -1 where
// no expert is left).  Every lane keeps PER keys, of experts lane, lane + 32, ...; topk times the
// warp takes the largest (lowest index among equals) and removes it, up to 4 keys per lane from
// sorted lists.
template <int PER>
__device__ __forceinline__ void topk_token(const RouteLaunch& L, int64_t m, int lane, int& id,
                                           float& w) {
  uint32_t key[PER];
  float mx = -INFINITY;
  auto logit = [&](int e) { return load_logit(L.logits, L.bf16, m * L.ld + e); };
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = i * 32 + lane;
    const float l = e < L.E ? logit(e) : -INFINITY;
    // the sigmoid grows with the logit, so without a bias the logits give the order (in fp32 the
    // sigmoids of different logits may be equal)
    float sc = l;
    if (L.scoring == 1 && L.bias) {
      sc = 1.0f / (1.0f + expf(-sc));
      if (e < L.E) sc += L.bias[e];
    }
    key[i] = l == -INFINITY ? 0u : score_key(sc);
    mx = fmaxf(mx, l);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  // softmax over all experts: only where the weights are not divided by their own sum
  float sum = 1.0f;
  if (L.scoring == 0 && !L.renormalize) {
    sum = 0.0f;
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (i * 32 + lane < L.E) {
        const float l = logit(i * 32 + lane);
        if (l != -INFINITY) sum += expf(l - mx);
      }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  }
  id = -1;
  constexpr bool kSorted = PER <= 4;
  uint32_t place[PER];
  if constexpr (kSorted) sort_keys<PER>(key, place);
  for (int j = 0; j < L.topk; ++j) {
    uint32_t best = 0;
    int at = 0x7FFFFFFF;
    if constexpr (kSorted) {
      best = key[0];
      at = (int)place[0] + lane;
    } else {
#pragma unroll
      for (int i = 0; i < PER; ++i)
        if (key[i] > best) {
          best = key[i];
          at = i * 32 + lane;
        }
    }
    const uint32_t top = __reduce_max_sync(0xffffffffu, best);
    if (top == 0) break;
    const int e = __reduce_min_sync(0xffffffffu, best == top ? at : 0x7FFFFFFF);
    if constexpr (kSorted) {
      const bool mine = at == e;
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        key[i] = !mine ? key[i] : i + 1 < PER ? key[i + 1] : 0u;
        if (i + 1 < PER) place[i] = mine ? place[i + 1] : place[i];
      }
    } else {
#pragma unroll
      for (int i = 0; i < PER; ++i)
        if (i * 32 + lane == e) key[i] = 0;
    }
    if (lane == j) id = e;
  }
  w = 0.0f;
  if (id >= 0) {
    const float l = logit(id);
    w = L.scoring == 1 ? 1.0f / (1.0f + expf(-l)) : expf(l - mx) / sum;
  }
  if (L.renormalize) {
    float s = w;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (id >= 0 && s != 0.0f) w /= s;  // all weights 0 stay 0
  }
  w *= L.scale;
}

__device__ __forceinline__ int group_of_id(int id, int E) { return id >= 0 && id < E ? id : E; }

// A block's exclusive scan of v[0 .. n) in shared memory, in place; T threads.
template <int T>
__device__ __forceinline__ void block_scan(int* v, int n, int* s_warp) {
  const int per = (n + T - 1) / T, b = (int)threadIdx.x * per, lane = threadIdx.x & 31;
  int sum = 0;
  for (int i = b; i < b + per && i < n; ++i) sum += v[i];
  int run = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, run, o);
    if (lane >= o) run += u;
  }
  if (lane == 31) s_warp[threadIdx.x >> 5] = run;
  __syncthreads();
  run -= sum;
  for (int w = 0; w < (int)(threadIdx.x >> 5); ++w) run += s_warp[w];
  for (int i = b; i < b + per && i < n; ++i) {
    const int x = v[i];
    v[i] = run;
    run += x;
  }
  __syncthreads();
}

// Stable places of a block's pairs [p0, p1): warp w takes a run of `run` pairs (a multiple of 32),
// counts per group its own pairs in order, the warps' counts are summed in warp order behind
// base[group], and each pair goes to base + earlier warps' + its rank in the warp.
template <int T, typename Count>
__device__ __forceinline__ void place_pairs(const int32_t* ids, int64_t p0, int64_t p1, int E,
                                            const int* base, Count* wc, int32_t* order) {
  constexpr int W = T / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, GE = E + 1;
  const int64_t run = ((p1 - p0 + T - 1) / T) * 32;
  const int64_t w0 = p0 + warp * run, w1 = w0 + run < p1 ? w0 + run : p1;
  for (int i = threadIdx.x; i < W * GE; i += T) wc[i] = 0;
  __syncthreads();
  Count* mine = wc + warp * GE;
#pragma unroll 1
  for (int pass = 0; pass < 2; ++pass) {
    for (int64_t q = w0; q < w1; q += 32) {
      const int64_t i = q + lane;
      const int e = i < w1 ? group_of_id(ids[i], E) : -1;
      const uint32_t same = __match_any_sync(0xffffffffu, e);
      const int rank = __popc(same & ((1u << lane) - 1u));
      const int before = e >= 0 ? mine[e] : 0;
      __syncwarp();
      if (e >= 0) {
        if (rank == 0) mine[e] = (Count)(before + __popc(same));
        if (pass) order[base[e] + before + rank] = (int32_t)i;
      }
      __syncwarp();
    }
    if (pass == 0) {
      __syncthreads();
      for (int e = threadIdx.x; e < GE; e += T) {
        int sum = 0;
        for (int w = 0; w < W; ++w) {
          const int c = (int)wc[w * GE + e];
          wc[w * GE + e] = (Count)sum;
          sum += c;
        }
      }
      __syncthreads();
    }
  }
}

// Everything in one block: few pairs, where a launch costs more than the work.  With logits while
// every token has a warp of its own (32 tokens: 6.6 us; 64 tokens, two rounds: 10.1, 8.0 in two launches;
// 128: 17.2 and 8.2), given ids up to 1024 pairs (1024: 5.0 us and 5.2; 2048: 7.1 and 5.5).
constexpr int64_t kOnePairs = 1024, kOneTokens = 32;
inline bool one_block(bool logits, int64_t M, int64_t pairs) {
  return pairs <= kOnePairs && (!logits || M <= kOneTokens);
}
template <int T>
inline size_t one_smem(int E) { return (size_t)(E + 1) * (4 + T / 32 * 2) + 16; }

// T = 256 up to 8 tokens (a warp each; 4.7 us, 5.3 with 1024 threads, whose barriers and sum over the
// warps' counts cost more) and given ids; 1024 for more tokens (16: 5.5 us, 6.7 with 256).  One block
// per SM is all there is, and saying so lets the compiler take the registers that it needs (16
// tokens, 256 experts, replayed from a graph: 7.4 us, 7.8 where it spilled some instead).
template <int PER, int kOneThreads>
__global__ void __launch_bounds__(kOneThreads, 1) k_route_one(const RouteLaunch L) {
  extern __shared__ int s_dyn[];
  __shared__ int s_warp[kOneThreads / 32], s_ids[kOnePairs];
  int* total = s_dyn;  // [E + 1]
  uint16_t* wc = reinterpret_cast<uint16_t*>(s_dyn + L.E + 1);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, P = (int)L.M * L.topk;
  for (int e = threadIdx.x; e <= L.E; e += kOneThreads) total[e] = 0;
  pdl_wait();
  pdl_launch_dependents();
  __syncthreads();
  if (L.logits) {
    for (int m = warp; m < L.M; m += kOneThreads / 32) {
      int id;
      float w;
      topk_token<PER>(L, m, lane, id, w);
      if (lane < L.topk) {
        L.ids[m * L.topk + lane] = id;
        L.weights[m * L.topk + lane] = w;
        s_ids[m * L.topk + lane] = id;
        atomicAdd(total + group_of_id(id, L.E), 1);
      }
    }
  } else {
    for (int i = threadIdx.x; i < P; i += kOneThreads) {
      s_ids[i] = L.ids[i];
      atomicAdd(total + group_of_id(s_ids[i], L.E), 1);
    }
  }
  __syncthreads();
  block_scan<kOneThreads>(total, L.E + 1, s_warp);
  for (int e = threadIdx.x; e <= L.E; e += kOneThreads) L.offsets[e] = total[e];
  place_pairs<kOneThreads>(s_ids, 0, P, L.E, total, wc, L.order);
}

// Many pairs: block c counts its run of pairs per group (after choosing them, where there are
// logits); a second launch sums the blocks' counts and places the pairs.
constexpr int kPlaceThreads = 512;
constexpr int kManyBlocks = 152;

template <int PER, int T>
__global__ void __launch_bounds__(T) k_route_count(const RouteLaunch L, int* hist) {
  __shared__ int s_count[kMaxGroups + 1];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int e = threadIdx.x; e <= L.E; e += T) s_count[e] = 0;
  pdl_wait();
  pdl_launch_dependents();
  __syncthreads();
  const int64_t m0 = blockIdx.x * L.block_tokens, m1 = min(m0 + L.block_tokens, L.M);
  if (L.logits) {
    for (int64_t m = m0 + warp; m < m1; m += T / 32) {
      int id;
      float w;
      topk_token<PER>(L, m, lane, id, w);
      if (lane < L.topk) {
        L.ids[m * L.topk + lane] = id;
        L.weights[m * L.topk + lane] = w;
        atomicAdd(s_count + group_of_id(id, L.E), 1);
      }
    }
  } else {
    for (int64_t i = m0 * L.topk + threadIdx.x; i < m1 * L.topk; i += T)
      atomicAdd(s_count + group_of_id(L.ids[i], L.E), 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e <= L.E; e += T) hist[blockIdx.x * (L.E + 1) + e] = s_count[e];
}

// More than half of an SM's shared memory, so that the placing blocks spread over the SMs: as they
// launch while the counting blocks run, four of them would go to the first SM that frees up (8192
// tokens, 8 of 128 experts: 25.0 us, 17.4 us spread out).
constexpr size_t kManySmem = 116 * 1024;
static_assert((kMaxGroups + 1) * (8 + kPlaceThreads / 32 * 4) <= kManySmem);

__global__ void __launch_bounds__(kPlaceThreads) k_route_place(const RouteLaunch L, const int* hist) {
  extern __shared__ int s_dyn[];
  __shared__ int s_warp[kPlaceThreads / 32];
  int* total = s_dyn;                // [E + 1]
  int* before = total + L.E + 1;     // [E + 1] of the blocks before this one
  uint32_t* wc = reinterpret_cast<uint32_t*>(before + L.E + 1);
  const int GE = L.E + 1;
  for (int e = threadIdx.x; e < GE; e += kPlaceThreads) total[e] = before[e] = 0;
  pdl_wait();
  pdl_launch_dependents();
  __syncthreads();
  const int all = (int)gridDim.x * GE, mine = (int)blockIdx.x * GE;
  int e = (int)threadIdx.x % GE;
  const int step = kPlaceThreads % GE;
#pragma unroll 8
  for (int i = threadIdx.x; i < all; i += kPlaceThreads) {
    const int v = __ldcg(hist + i);
    if (v) {
      atomicAdd(total + e, v);
      if (i < mine) atomicAdd(before + e, v);
    }
    e += step;
    if (e >= GE) e -= GE;
  }
  __syncthreads();
  block_scan<kPlaceThreads>(total, GE, s_warp);
  if (blockIdx.x == 0)
    for (int e = threadIdx.x; e < GE; e += kPlaceThreads) L.offsets[e] = total[e];
  for (int e = threadIdx.x; e < GE; e += kPlaceThreads) before[e] += total[e];
  __syncthreads();
  const int64_t m0 = blockIdx.x * L.block_tokens, m1 = min(m0 + L.block_tokens, L.M);
  if (m0 < m1) place_pairs<kPlaceThreads>(L.ids, m0 * L.topk, m1 * L.topk, L.E, before, wc, L.order);
}

template <typename F>
cudaError_t launch_pdl(F f, int grid, int threads, size_t smem, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return f(cfg);
}

template <int PER, int T>
cudaError_t route_one(const RouteLaunch& L, cudaStream_t s) {
  static int done[64] = {0};
  const cudaError_t e = set_up_kernel(k_route_one<PER, T>, one_smem<T>(kMaxGroups), done);
  if (e != cudaSuccess) return e;
  return launch_pdl([&](const cudaLaunchConfig_t& c) { return cudaLaunchKernelEx(&c, k_route_one<PER, T>, L); },
                    1, T, one_smem<T>(L.E), s);
}

template <int PER>
cudaError_t route_per(RouteLaunch L, cudaStream_t s) {
  const int64_t P = L.M * L.topk;
  if (one_block(L.logits != nullptr, L.M, P))
    return !L.logits || L.M <= 8 ? route_one<PER, 256>(L, s) : route_one<PER, 1024>(L, s);
  static int done[64] = {0};
  cudaError_t e = set_up_kernel(k_route_place, kManySmem, done);
  if (e != cudaSuccess) return e;
  int* hist = reinterpret_cast<int*>(reinterpret_cast<uint8_t*>(L.workspace) + 256);
  const int64_t want = L.logits ? (L.M + 31) / 32 : (P + 255) / 256;
  const int blocks = (int)(want < kManyBlocks ? want : kManyBlocks);
  L.block_tokens = (L.M + blocks - 1) / blocks;
  constexpr int T = PER > 8 ? 512 : 1024;  // registers for the keys (8192 tokens: 9.0 us, 11.7 with 512)
  e = launch_pdl(
      [&](const cudaLaunchConfig_t& c) { return cudaLaunchKernelEx(&c, k_route_count<PER, T>, L, hist); },
      blocks, T, 0, s);
  if (e != cudaSuccess) return e;
  return launch_pdl(
      [&](const cudaLaunchConfig_t& c) { return cudaLaunchKernelEx(&c, k_route_place, L, (const int*)hist); },
      blocks, kPlaceThreads, kManySmem, s);
}

}  // namespace

size_t route_workspace_bytes(int64_t pairs, int64_t E) {
  if (pairs <= kOneTokens) return 256;  // one block with logits too, whatever topk
  return 256 + ((size_t)kManyBlocks * (E + 1) * 4 + 255) / 256 * 256;
}

cudaError_t launch_route(const RouteLaunch& L, cudaStream_t s) {
  if (L.E <= 32 || !L.logits) return route_per<1>(L, s);
  if (L.E <= 128) return route_per<4>(L, s);
  if (L.E <= 256) return route_per<8>(L, s);
  return route_per<32>(L, s);
}

}  // namespace vt
