// Low-rank adapters of many requests beside a shared projection:
//   out[m] = y[m] + scale[a] * B_a (A_a x[m]),  a the adapter of row m's group.
#include <cuda_bf16.h>

#include "common.cuh"
#include "kernels.h"

namespace vt {

namespace {

// One cluster of kCluster CTAs per tile of up to TM rows of one adapter.  First each CTA sums its
// share of K (v = A x, ranks as the MMA's rows, tokens as its columns) and the cluster adds the
// shares through distributed shared memory, in CTA order; then each CTA does its share of N
// (tokens as rows, columns of B as columns) and adds it to y.  x, y and out cross the memory bus
// once, an adapter once per tile (from L2 after the first).  v is fp32; as an MMA operand it is
// the sum of two bf16 values (16 significant bits).
// Within a block of 32 k (or ranks) lane t of a quad holds the 8 physical positions 8t .. 8t + 7,
// one 16-byte load, in the MMA's k columns {2t, 2t+1, 2t+8, 2t+9} of two steps; both operands use
// the same order, so the products are those of the physical order.
constexpr int kCluster = 8;
constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;

__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The float at shared-memory address `addr` of CTA `rank` of the cluster.
__device__ __forceinline__ float4 ld_cluster_v4(uint32_t addr, uint32_t rank) {
  uint32_t a;
  float4 v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(addr), "r"(rank));
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(a));
  return v;
}

// 8 consecutive 16-bit values, the first `n` of them valid (the others 0); `vec`: 16-byte aligned.
__device__ __forceinline__ uint4 load8(const __nv_bfloat16* p, int64_t n, bool vec) {
  if (vec && n >= 8) return __ldg(reinterpret_cast<const uint4*>(p));
  uint32_t w[4] = {0, 0, 0, 0};
  const uint16_t* q = reinterpret_cast<const uint16_t*>(p);
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < n) w[i >> 1] |= (uint32_t)__ldg(q + i) << ((i & 1) * 16);
  return make_uint4(w[0], w[1], w[2], w[3]);
}

struct LoraParams {
  LoraLaunch L;
  int vec_x, vec_a, vec_b, vec_y;  // 16-byte aligned rows
};

// RM: ranks held (16 .. RM per adapter).
template <int TM, int RM>
struct LoraSmem {
  static constexpr int WT = TM / 16, WK = kWarps / WT;      // token groups, shares of the CTA's k
  static constexpr int VStride = RM + 4;                    // floats per token of the partial sums
  static constexpr int HStride = RM + 8;                    // bf16 per token of v's two terms
  static constexpr int Partial = WK * TM * VStride * 4;
  static constexpr int Halves = 2 * TM * HStride * 2;
  static constexpr int Bytes = Partial + Halves;
};

template <int TM, int RM>
__global__ void __launch_bounds__(kThreads) k_lora(const LoraParams p) {
  using S = LoraSmem<TM, RM>;
  const LoraLaunch& L = p.L;
  extern __shared__ __align__(16) uint8_t smem[];
  float* s_part = reinterpret_cast<float*>(smem);                        // [WK][TM][VStride]
  __nv_bfloat16* s_hi = reinterpret_cast<__nv_bfloat16*>(smem + S::Partial);  // [TM][HStride]
  __nv_bfloat16* s_lo = s_hi + TM * S::HStride;
  __shared__ int s_warp[kWarps], s_e, s_i0, s_n, s_row[TM];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  const int rank = (int)cluster_rank();
  const int tile = (int)(blockIdx.x / kCluster);
  pdl_wait();
  pdl_launch_dependents();

  // the tile's group: prefix sums of the groups' tiles; group L.L holds the rows without adapter
  if (tid == 0) s_e = -1;
  {
    constexpr int per = (kMaxGroups + 1 + kThreads - 1) / kThreads;
    int b[per + 1], nt[per], sum = 0;
    const int e0 = tid * per;
#pragma unroll
    for (int i = 0; i <= per; ++i) {
      const int e = e0 + i;
      int v = e <= L.L ? __ldcg(L.offsets + e) : (int)L.M;
      b[i] = v < 0 ? 0 : (v > (int)L.M ? (int)L.M : v);
    }
#pragma unroll
    for (int i = 0; i < per; ++i) {
      const int n = b[i + 1] - b[i];
      nt[i] = e0 + i <= L.L && n > 0 ? (n + TM - 1) / TM : 0;
      sum += nt[i];
    }
    int run = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, run, o);
      if (lane >= o) run += u;
    }
    if (lane == 31) s_warp[warp] = run;
    __syncthreads();
    run -= sum;
    for (int w = 0; w < warp; ++w) run += s_warp[w];
#pragma unroll
    for (int i = 0; i < per; ++i) {
      if (tile >= run && tile < run + nt[i]) {
        s_e = e0 + i;
        s_i0 = b[i] + (tile - run) * TM;
        s_n = min(TM, b[i + 1] - s_i0);
      }
      run += nt[i];
    }
  }
  __syncthreads();
  const int e = s_e, n = s_n;
  if (e < 0) return;  // the whole cluster: no such tile
  if (e == L.L && L.out == L.y) return;
  if (tid < TM) {
    int r = -1;
    if (tid < n) {
      r = __ldcg(L.order + s_i0 + tid);
      if (r < 0 || r >= L.M) r = -1;
    }
    s_row[tid] = r;
  }
  int R = 0;
  if (e < L.L) R = L.ranks ? min(max(__ldg(L.ranks + e), 0), L.R) : L.R;
  __syncthreads();
  const __nv_bfloat16* y = reinterpret_cast<const __nv_bfloat16*>(L.y);
  __nv_bfloat16* out = reinterpret_cast<__nv_bfloat16*>(L.out);

  if (R > 0) {
    // ---------------------------------------------------------- v = A x, this CTA's k
    const int wt = warp % S::WT, wk = warp / S::WT;
    const int64_t kb = (L.K + 31) / 32;
    const int64_t k0 = kb * rank / kCluster, k1 = kb * (rank + 1) / kCluster;
    const __nv_bfloat16* A = reinterpret_cast<const __nv_bfloat16*>(L.A) + (int64_t)e * L.R * L.K;
    const __nv_bfloat16* x = reinterpret_cast<const __nv_bfloat16*>(L.x);
    float acc[RM / 16][2][4] = {};
    int row[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) row[j] = s_row[wt * 16 + j * 8 + g];
    if (wt * 16 < n) {
#pragma unroll 2
      for (int64_t b = k0 + wk; b < k1; b += S::WK) {
        const int64_t k = b * 32 + t * 8, left = L.K - k;
        uint4 xv[2];
#pragma unroll
        for (int j = 0; j < 2; ++j)
          xv[j] = row[j] >= 0 ? load8(x + row[j] * L.ldx + k, left, p.vec_x) : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int m = 0; m < RM / 16; ++m) {
          if (m * 16 >= R) break;
          uint4 a0 = make_uint4(0, 0, 0, 0), a1 = a0;
          if (m * 16 + g < R) a0 = load8(A + (int64_t)(m * 16 + g) * L.K + k, left, p.vec_a);
          if (m * 16 + g + 8 < R) a1 = load8(A + (int64_t)(m * 16 + g + 8) * L.K + k, left, p.vec_a);
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            mma_bf16(acc[m][j], a0.x, a1.x, a0.y, a1.y, xv[j].x, xv[j].y);
            mma_bf16(acc[m][j], a0.z, a1.z, a0.w, a1.w, xv[j].z, xv[j].w);
          }
        }
      }
    }
    // rows of the MMA are ranks, columns tokens
#pragma unroll
    for (int m = 0; m < RM / 16; ++m)
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          s_part[(wk * TM + wt * 16 + j * 8 + 2 * t + (i & 1)) * S::VStride + m * 16 + g + (i >> 1) * 8] =
              acc[m][j][i];
    __syncthreads();
    // the CTA's share of v, over its warps' shares of k
    for (int i = tid; i < TM * RM / 4; i += kThreads) {
      const int tok = i / (RM / 4), r4 = i % (RM / 4) * 4;
      float4 v = *reinterpret_cast<float4*>(s_part + tok * S::VStride + r4);
#pragma unroll
      for (int w = 1; w < S::WK; ++w) {
        const float4 u = *reinterpret_cast<float4*>(s_part + (w * TM + tok) * S::VStride + r4);
        v.x += u.x; v.y += u.y; v.z += u.z; v.w += u.w;
      }
      *reinterpret_cast<float4*>(s_part + tok * S::VStride + r4) = v;
    }
    cluster_arrive();
    cluster_wait();
    // v over the cluster's CTAs, times the adapter's scale, as two bf16 terms
    const float scale = __ldg(L.scale + e);
    for (int i = tid; i < TM * RM / 4; i += kThreads) {
      const int tok = i / (RM / 4), r4 = i % (RM / 4) * 4;
      float4 v = make_float4(0, 0, 0, 0);
      if (tok < n && r4 < R) {
        const uint32_t at = smem_u32(s_part + tok * S::VStride + r4);
#pragma unroll
        for (int c = 0; c < kCluster; ++c) {
          const float4 u = ld_cluster_v4(at, c);
          v.x += u.x; v.y += u.y; v.z += u.z; v.w += u.w;
        }
      }
      const float f[4] = {v.x * scale, v.y * scale, v.z * scale, v.w * scale};
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const __nv_bfloat16 h = __float2bfloat16_rn(f[c]);
        s_hi[tok * S::HStride + r4 + c] = h;
        // an infinite or NaN v is all in its first term
        const float d = f[c] - __bfloat162float(h);
        s_lo[tok * S::HStride + r4 + c] = __float2bfloat16_rn(isfinite(f[c]) ? d : 0.0f);
      }
    }
    cluster_arrive();  // no CTA may leave while another reads its shared memory: waited for below
    __syncthreads();
  }

  // -------------------------------------------------------- out = y + v B^T, this CTA's columns
  const int64_t nb = (L.N + 31) / 32;
  const int64_t n0 = nb * rank / kCluster, n1 = nb * (rank + 1) / kCluster;
  const __nv_bfloat16* B = reinterpret_cast<const __nv_bfloat16*>(L.B) + (int64_t)(R > 0 ? e : 0) * L.N * L.R;
  for (int64_t b = n0 + warp; b < n1; b += kWarps) {
    // tile j of four, MMA column c: physical column 32b + 8 (c / 2) + 2j + c % 2, so that lane t
    // ends with the 8 columns from 32b + 8t on
    uint4 bv[RM / 32 > 0 ? RM / 32 : 1][4];
#pragma unroll
    for (int q = 0; q < RM / 32; ++q)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int64_t col = b * 32 + 8 * (g >> 1) + 2 * j + (g & 1);
        bv[q][j] = make_uint4(0, 0, 0, 0);
        if (col < L.N && q * 32 + t * 8 < R)
          bv[q][j] = load8(B + col * L.R + q * 32 + t * 8, R - (q * 32 + t * 8), p.vec_b);
      }
    const int64_t c0 = b * 32 + t * 8, left = L.N - c0;
#pragma unroll 1
    for (int m = 0; m * 16 < n; ++m) {
      float d[4][4] = {};
      uint4 yv[2];
      int row[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        row[h] = s_row[m * 16 + h * 8 + g];
        yv[h] = make_uint4(0, 0, 0, 0);
        if (row[h] >= 0 && left > 0) {
          // out may be y itself: not the read-only path
          const __nv_bfloat16* src = y + row[h] * L.ldy + c0;
          if (p.vec_y && left >= 8) {
            yv[h] = *reinterpret_cast<const uint4*>(src);
          } else {
            uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
            for (int i = 0; i < 8; ++i)
              if (i < left) w[i >> 1] |= (uint32_t)reinterpret_cast<const uint16_t*>(src)[i] << ((i & 1) * 16);
            yv[h] = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
      }
      if (R > 0) {
#pragma unroll
        for (int q = 0; q < RM / 32; ++q) {
          if (q * 32 >= R) break;
#pragma unroll
          for (int part = 0; part < 2; ++part) {
            const __nv_bfloat16* s = (part ? s_lo : s_hi) + (m * 16 + g) * S::HStride + q * 32 + t * 8;
            const uint4 v0 = *reinterpret_cast<const uint4*>(s);
            const uint4 v1 = *reinterpret_cast<const uint4*>(s + 8 * S::HStride);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              mma_bf16(d[j], v0.x, v1.x, v0.y, v1.y, bv[q][j].x, bv[q][j].y);
              mma_bf16(d[j], v0.z, v1.z, v0.w, v1.w, bv[q][j].z, bv[q][j].w);
            }
          }
        }
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (row[h] < 0 || left <= 0) continue;
        const uint32_t w[4] = {yv[h].x, yv[h].y, yv[h].z, yv[h].w};
        uint32_t o[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const __nv_bfloat162 z = __floats2bfloat162_rn(__uint_as_float(w[j] << 16) + d[j][2 * h],
                                                         __uint_as_float(w[j] & 0xFFFF0000u) + d[j][2 * h + 1]);
          o[j] = *reinterpret_cast<const uint32_t*>(&z);
        }
        __nv_bfloat16* dst = out + row[h] * L.ldo + c0;
        if (p.vec_y && left >= 8) {
          *reinterpret_cast<uint4*>(dst) = make_uint4(o[0], o[1], o[2], o[3]);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (i < left) reinterpret_cast<uint16_t*>(dst)[i] = (uint16_t)(o[i >> 1] >> ((i & 1) * 16));
        }
      }
    }
  }
  if (R > 0) cluster_wait();
}

template <int TM, int RM>
cudaError_t launch(const LoraParams& p, cudaStream_t s) {
  constexpr int bytes = LoraSmem<TM, RM>::Bytes;
  static int done[64] = {0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!done[dev]) {
    e = cudaFuncSetAttribute(k_lora<TM, RM>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    done[dev] = 1;
  }
  // at most one partial tile per group in use, the rows without adapter a group too
  const int64_t groups = p.L.M < p.L.L + 1 ? p.L.M : p.L.L + 1;
  const int64_t tiles = groups + p.L.M / TM;
  if (tiles * kCluster > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(tiles * kCluster));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = bytes;
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = kCluster;
  at[1].val.clusterDim.y = 1;
  at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, k_lora<TM, RM>, p);
}

template <int RM>
cudaError_t launch_rank(const LoraParams& p, cudaStream_t s) {
  // long runs of one adapter: tiles of 64 rows read the adapter a quarter as often
  return p.L.M >= 24 * (int64_t)p.L.L ? launch<64, RM>(p, s) : launch<16, RM>(p, s);
}

}  // namespace

cudaError_t launch_lora(const LoraLaunch& L, cudaStream_t s) {
  LoraParams p;
  p.L = L;
  p.vec_x = (uintptr_t)L.x % 16 == 0 && L.ldx % 8 == 0;
  p.vec_a = (uintptr_t)L.A % 16 == 0 && L.K % 8 == 0;
  p.vec_b = (uintptr_t)L.B % 16 == 0 && L.R % 8 == 0;
  p.vec_y = (uintptr_t)L.y % 16 == 0 && L.ldy % 8 == 0 && (uintptr_t)L.out % 16 == 0 && L.ldo % 8 == 0;
  if (L.R <= 32) return launch_rank<32>(p, s);
  if (L.R <= 64) return launch_rank<64>(p, s);
  return launch_rank<128>(p, s);
}

}  // namespace vt
