// Low-rank adapters of many requests beside a shared projection:
//   out[m] = y[m] + scale[a] * B_a (A_a x[m]),  a the adapter of row m's group.
#include <cuda_bf16.h>

#include "common.cuh"
#include "handle.h"
#include "kernels.h"

namespace vt {

namespace {

// One cluster of 8 or 16 CTAs per tile of up to TM rows of one adapter.  First each CTA sums its
// share of K (v = A x: ranks are the MMA's rows, tokens its columns) and the cluster adds the
// shares through distributed shared memory, in CTA order; then each CTA adds v B^T to its share of
// y's columns (tokens are rows).  x, y and out cross the memory bus once, an adapter once per tile
// (from L2 after the first), no workspace, one launch.  v is fp32; as an MMA operand it is the sum
// of two bf16 values (16 significant bits).
// Memory bounds it, so everything streams through a ring of shared-memory chunks filled by
// asynchronous 16-byte copies, the columns' chunks already under way while v is exchanged (with
// loads to registers too few bytes were in flight: 53 us for 5003 rows, 4096 -> 5120, rank 32,
// 44 to 49 with them, from card to card).  Rows of y that are not whole 16-byte pieces (odd N) are copied from the boundary
// before them on (3000 rows, 4096 -> 4095: 49 us, 92 value by value; 30 for 4096 columns); such rows of
// x, A and B value by value.
constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;

// TM: rows per tile; RM: ranks held.  A chunk has a fixed cost of barriers and copies to issue:
// 256 wide where a CTA has an SM for itself (1 row: 4.6 us, 5.3 with 128); else 128 and as many CTAs
// per SM as hold two chunks each, with 80 registers a thread for three (96 rows of 64 adapters:
// 19.8 us; two CTAs of four chunks 20.5; three of five chunks of 64 22.3).
template <int TM, int RM, int kCluster>
struct LoraSmem {
  static constexpr int kChunk = kCluster == 16 ? 256 : 128;  // k, or columns, per chunk
  static constexpr int kStride = kChunk * 2 + 16;           // bytes per row of x, A or y (no bank conflicts)
  // v's warps: WT groups of 16 tokens, WR of rank tiles (each takes every WR-th), WK shares of k
  static constexpr int WT = TM / 16, WR = RM / 16 < kWarps / WT ? RM / 16 : kWarps / WT;
  static constexpr int WK = kWarps / WT / WR;
  static constexpr int BStride = RM * 2 + 16;               // bytes per column of B, per row of v
  static constexpr int ChunkA = (RM + TM) * kStride, ChunkB = kChunk * BStride + TM * kStride;
  static constexpr int Stage = ChunkA > ChunkB ? ChunkA : ChunkB;
  static constexpr int VStride = RM + 4;                    // floats per token of the partial sums
  static constexpr int Partial = WK * TM * VStride * 4, V = 2 * TM * BStride;
  static constexpr int stages(int ctas) { return ((228 / ctas - 1) * 1024 - 512 - Partial - V) / Stage; }
  static constexpr int Ctas = kCluster == 16 ? 1
                              : TM == 16     ? (stages(3) >= 2 ? 3 : stages(2) >= 2 ? 2 : 1)
                                             : (stages(2) >= 3 ? 2 : 1);
  static constexpr int Stages = stages(Ctas) < 6 ? stages(Ctas) : 6;
  static constexpr int OffPart = Stages * Stage, OffV = OffPart + Partial;
  static constexpr int Bytes = OffV + V;
  static_assert(Stages >= 2, "shared memory");
};

__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void ldmatrix4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
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
// Four floats at shared-memory address `addr` of CTA `rank` of the cluster.
__device__ __forceinline__ float4 ld_cluster_v4(uint32_t addr, uint32_t rank) {
  uint32_t a;
  float4 v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(addr), "r"(rank));
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(a));
  return v;
}

__device__ __forceinline__ void st_cluster_v2(uint32_t addr, uint32_t rank, uint2 v) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(addr), "r"(rank));
  asm volatile("st.shared::cluster.v2.b32 [%0], {%1, %2};" ::"r"(a), "r"(v.x), "r"(v.y) : "memory");
}

// Four 16-bit values from any place in shared memory.
__device__ __forceinline__ uint2 ld_shared_4h(uint32_t addr) {
  uint16_t v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v[i]) : "r"(addr + 2 * i) : "memory");
  return make_uint2(v[0] | (uint32_t)v[1] << 16, v[2] | (uint32_t)v[3] << 16);
}

// 8 consecutive values to shared memory, the first n (0 to 8) of them valid (the others zeros).  VEC: one
// asynchronous copy (src 16-byte aligned); else value by value.
template <bool VEC>
__device__ __forceinline__ void copy8(uint32_t dst, const __nv_bfloat16* src, int n) {
  if constexpr (VEC) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n * 2)
                 : "memory");
  } else {
    uint32_t w[4] = {0, 0, 0, 0};
    const uint16_t* q = reinterpret_cast<const uint16_t*>(src);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) w[i >> 1] |= (uint32_t)q[i] << ((i & 1) * 16);
    st_shared_v4(dst, w[0], w[1], w[2], w[3]);
  }
}

// VEC: the rows of x, A and B are whole 16-byte pieces; VECY: those of y and out too.
template <int TM, int RM, int kCluster, bool VEC, bool VECY>
__global__ void __launch_bounds__(kThreads, LoraSmem<TM, RM, kCluster>::Ctas) k_lora(const LoraLaunch L) {
  using S = LoraSmem<TM, RM, kCluster>;
  constexpr int kChunk = S::kChunk, kStride = S::kStride;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ int s_warp[kWarps], s_e, s_i0, s_n, s_row[TM];
  const uint32_t ring = smem_u32(smem);
  float* s_part = reinterpret_cast<float*>(smem + S::OffPart);  // [WK][TM][VStride]
  const uint32_t v_hi = ring + S::OffV, v_lo = v_hi + TM * S::BStride;
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

  // this CTA's k and columns, in blocks of 32
  const int K = (int)L.K, N = (int)L.N, R16 = (R + 15) & ~15;
  const int kb = (K + 31) / 32, nb = (N + 31) / 32;
  const int k0 = kb * rank / kCluster * 32, k1 = R ? min(kb * (rank + 1) / kCluster * 32, K) : k0;
  const int c0 = nb * rank / kCluster * 32, c1 = min(nb * (rank + 1) / kCluster * 32, N);
  const int nk = (k1 - k0 + kChunk - 1) / kChunk, chunks = nk + (c1 - c0 + kChunk - 1) / kChunk;
  const __nv_bfloat16* A = reinterpret_cast<const __nv_bfloat16*>(L.A) + (R ? (int64_t)e * L.R * K : 0);
  const __nv_bfloat16* B = reinterpret_cast<const __nv_bfloat16*>(L.B) + (R ? (int64_t)e * N * L.R : 0);
  const __nv_bfloat16* x = reinterpret_cast<const __nv_bfloat16*>(L.x);
  const __nv_bfloat16* y = reinterpret_cast<const __nv_bfloat16*>(L.y);

  // Chunk c of the CTA's work: nk of x [TM] over A [R16] (rows of 128 k), then y [TM] over B
  // [128 columns] (rows of ranks).  A thread copies piece `pc` of rows r0, r0 + RP, ... of x, y and
  // A, and piece bp of columns bc0, bc0 + bstep, ... of B, 2^sh >= R16 / 8 threads to a column; its
  // pointers move on by a chunk per fetch (issuing the copies is a good part of a chunk's time).
  // Sources of zeros point at valid memory all the same.
  constexpr int P = kChunk / 8, RP = kThreads / P, XP = TM / RP;  // pieces per row, rows per pass
  const int pc = tid % P, r0 = tid / P;
  const __nv_bfloat16* px[XP];  // this thread's pieces of x, then of y
  int xrow[XP];
#pragma unroll
  for (int i = 0; i < XP; ++i) {
    xrow[i] = s_row[r0 + i * RP];
    px[i] = x + max(xrow[i], 0) * L.ldx + k0 + pc * 8;
  }
  const int sh = R16 <= 16 ? 1 : R16 <= 32 ? 2 : R16 <= 64 ? 3 : 4;
  const int bp = tid & ((1 << sh) - 1), bc0 = tid >> sh, bstep = kThreads >> sh;
  const int have = min(max(R - bp * 8, 0), 8);  // ranks of this thread's piece of a column
  const int64_t stepA = (int64_t)RP * K, stepB = (int64_t)bstep * L.R;
  const __nv_bfloat16* pa = A + (int64_t)r0 * K + k0 + pc * 8;
  const __nv_bfloat16* pb = B + (int64_t)(c0 + bc0) * L.R + bp * 8;
  const uint32_t to_row = ring + r0 * kStride + pc * 16, to_b = ring + TM * kStride + bc0 * S::BStride + bp * 16;
  // y's rows without VECY, where VEC: the 16-byte pieces from the boundary before the row's first
  // column on, one more than the columns need (a row of a chunk has room for it; what lies beside the
  // columns is not used); y8: that column's place in the first piece
  constexpr bool kWindow = VEC && !VECY;
  int y8[kWindow ? XP : 1];
  int fetched = 0;
  uint32_t slot = 0;  // byte offset of the next chunk's stage
  auto fetch = [&] {
    const int c = fetched++;
    if (c < nk) {
      const int left = min(max(k1 - (k0 + c * kChunk + pc * 8), 0), 8);
      const uint32_t to = to_row + slot;
#pragma unroll
      for (int i = 0; i < XP; ++i) {
        if (i * RP < n) copy8<VEC>(to + i * RP * kStride, left > 0 ? px[i] : x, xrow[i] >= 0 ? left : 0);
        px[i] += kChunk;
      }
      const __nv_bfloat16* a = pa;
#pragma unroll
      for (int i = 0; i < (RM + RP - 1) / RP; ++i) {
        if (i * RP < R16) copy8<VEC>(to + (TM + i * RP) * kStride, left > 0 && r0 + i * RP < R ? a : A, r0 + i * RP < R ? left : 0);
        a += stepA;
      }
      pa += kChunk;
    } else if (c < chunks) {
      if (c == nk) {
#pragma unroll
        for (int i = 0; i < XP; ++i) {
          px[i] = y + max(xrow[i], 0) * L.ldy + c0;
          if constexpr (kWindow) {
            y8[i] = (int)((uintptr_t)px[i] >> 1) & 7;
            px[i] -= y8[i];
          }
          px[i] += pc * 8;
        }
      }
      const int b0 = c0 + (c - nk) * kChunk, left = min(max(c1 - (b0 + pc * 8), 0), 8);
      const uint32_t to = to_row + slot;
#pragma unroll
      for (int i = 0; i < XP; ++i) {
        if (i * RP < n) {
          const uint32_t dst = to + i * RP * kStride;
          if constexpr (kWindow) {
            const int ends = xrow[i] >= 0 ? min(kChunk, c1 - b0) + y8[i] - pc * 8 : 0;
            copy8<true>(dst, ends > 0 ? px[i] : A, min(max(ends, 0), 8));
            if (pc == P - 1) copy8<true>(dst + 16, ends > 8 ? px[i] + 8 : A, min(max(ends - 8, 0), 8));
          } else {
            copy8<VECY>(dst, left > 0 ? px[i] : y, xrow[i] >= 0 ? left : 0);
          }
        }
        px[i] += kChunk;
      }
      if (bp * 8 < R16) {
        uint32_t tb = to_b + slot;
        const __nv_bfloat16* b = pb;
        for (int j = bc0; j < kChunk; j += bstep) {
          const bool on = b0 + j < c1 && have > 0;
          copy8<VEC>(tb, on ? b : B, on ? have : 0);
          tb += bstep * S::BStride;
          b += stepB;
        }
        pb += (int64_t)kChunk * L.R;
      }
    }
    slot = slot + S::Stage == S::Stages * S::Stage ? 0 : slot + S::Stage;
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int c = 0; c < S::Stages - 1; ++c) fetch();
  // the ring's next chunk: landed for every thread, and the one before it used by every thread
  uint32_t used = 0;
  auto next = [&] {
    asm volatile("cp.async.wait_group %0;" ::"n"(S::Stages - 2) : "memory");
    __syncthreads();
    fetch();
    const uint32_t st = ring + used;
    used = used + S::Stage == S::Stages * S::Stage ? 0 : used + S::Stage;
    return st;
  };
  // rows of tokens past n in a chunk hold what earlier chunks left: finite or not, they are
  // columns (then rows) of their own that are not stored
  const int lrow = lane & 7, lmat = lane >> 3;  // this lane's row and matrix of an ldmatrix

  bool late_wait = false;
  if (R > 0) {
    // ---------------------------------------------------------------- v = A x
    const int wt = warp % S::WT, wr = warp / S::WT % S::WR, wk = warp / S::WT / S::WR;
    constexpr int MT = RM / 16 / S::WR;  // rank tiles wr, wr + WR, ... of the warp
    float acc[MT][2][4] = {};
    for (int c = 0; c < nk; ++c) {
      const uint32_t st = next();
      if (wt * 16 >= n || wr * 16 >= R) continue;
      // k steps wk, wk + WK, ...: the fragments of kS of them are loaded before their products
      constexpr int kSteps = kChunk / 16 / S::WK, kS = kSteps < 4 / MT ? kSteps : MT < 4 ? 4 / MT : 1;
#pragma unroll
      for (int s0 = 0; s0 < kSteps; s0 += kS) {
        uint32_t xv[kS][4], av[kS][MT][4];
#pragma unroll
        for (int s = 0; s < kS; ++s) {
          const int ks = ((s0 + s) * S::WK + wk) * 32;  // byte of the 16-k step in a row
          // tokens 0-7 (k low, high), 8-15
          ldmatrix4(st + (wt * 16 + (lmat >> 1) * 8 + lrow) * kStride + ks + (lmat & 1) * 16, xv[s]);
#pragma unroll
          for (int i = 0; i < MT; ++i) {
            const int m = i * S::WR + wr;
            if (m * 16 < R)
              ldmatrix4(st + (TM + m * 16 + (lmat & 1) * 8 + lrow) * kStride + ks + (lmat >> 1) * 16, av[s][i]);
          }
        }
#pragma unroll
        for (int s = 0; s < kS; ++s)
#pragma unroll
          for (int i = 0; i < MT; ++i)
            if ((i * S::WR + wr) * 16 < R) {
              mma_bf16(acc[i][0], av[s][i], xv[s][0], xv[s][1]);
              mma_bf16(acc[i][1], av[s][i], xv[s][2], xv[s][3]);
            }
      }
    }
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          s_part[(wk * TM + wt * 16 + j * 8 + 2 * t + (i & 1)) * S::VStride + (m * S::WR + wr) * 16 + g +
                 (i >> 1) * 8] = acc[m][j][i];
    const int r4s = R16 / 4;
    if constexpr (S::WK > 1) {  // the CTA's share of v, over its warps' shares of k
      __syncthreads();
      for (int i = tid; i < n * r4s; i += kThreads) {
        float* at = s_part + i / r4s * S::VStride + i % r4s * 4;
        float4 v = *reinterpret_cast<float4*>(at);
  #pragma unroll
        for (int w = 1; w < S::WK; ++w) {
          const float4 u = *reinterpret_cast<float4*>(at + w * TM * S::VStride);
          v.x += u.x; v.y += u.y; v.z += u.z; v.w += u.w;
        }
        *reinterpret_cast<float4*>(at) = v;
      }
    }
    cluster_arrive();
    cluster_wait();
    // v over the cluster's CTAs, times the adapter's scale, as two bf16 terms.  Large tiles: each
    // CTA sums its share of the values and writes it to all (one more barrier, an eighth of the
    // reads); small ones: each sums them all.  4096 -> 4096, shared and not: 16 groups of four values
    // 5.3 and 5.0 us, 64 groups 4.8 and 5.0, 128 groups 5.3 and 6.1; 5003 rows, 4096 -> 5120: 46 and 55.
    const float scale = __ldg(L.scale + e);
    const int entries = n * r4s;
    const bool share = entries >= kThreads / 4;
    const int i0 = share ? entries * rank / kCluster : 0, i1 = share ? entries * (rank + 1) / kCluster : entries;
    for (int i = i0 + tid; i < i1; i += kThreads) {
      const int tok = i / r4s, r4 = i % r4s * 4;
      const uint32_t at = smem_u32(s_part + tok * S::VStride + r4);
      float4 u[kCluster], v = make_float4(0, 0, 0, 0);
#pragma unroll
      for (int c = 0; c < kCluster; ++c) u[c] = ld_cluster_v4(at, c);
#pragma unroll
      for (int c = 0; c < kCluster; ++c) {
        v.x += u[c].x; v.y += u[c].y; v.z += u[c].z; v.w += u[c].w;
      }
      // ranks past R are zeros whatever x holds (an infinity times A's zeros there is NaN)
      const float f[4] = {r4 < R ? v.x * scale : 0.0f, r4 + 1 < R ? v.y * scale : 0.0f,
                          r4 + 2 < R ? v.z * scale : 0.0f, r4 + 3 < R ? v.w * scale : 0.0f};
      uint32_t h[4], l[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const __nv_bfloat16 hi = __float2bfloat16_rz(f[c]);  // (a rounded one could overflow)
        // Both terms have v's sign and neither is 0 unless v is, so that an infinite entry of B
        // gives infinities of one sign: an infinite v is in both terms, and the second term of a v
        // that the first one holds whole is 2^-24 of it (0 times infinity would be NaN).
        h[c] = __bfloat16_as_ushort(hi);
        l[c] = __bfloat16_as_ushort(__float2bfloat16_rn(isfinite(f[c]) ? f[c] - __bfloat162float(hi) : f[c]));
        if (!(l[c] & 0x7FFFu) && f[c] != 0.0f)
          l[c] = __bfloat16_as_ushort(__float2bfloat16_rn(copysignf(fmaxf(fabsf(f[c]) * 0x1p-24f, 0x1p-133f), f[c])));
      }
      const uint32_t to = tok * S::BStride + r4 * 2;
      const uint2 hv = make_uint2(h[0] | h[1] << 16, h[2] | h[3] << 16);
      const uint2 lv = make_uint2(l[0] | l[1] << 16, l[2] | l[3] << 16);
      if (share) {
#pragma unroll
        for (int c = 0; c < kCluster; ++c) {
          st_cluster_v2(v_hi + to, c, hv);
          st_cluster_v2(v_lo + to, c, lv);
        }
      } else {
        st_cluster_v2(v_hi + to, rank, hv);
        st_cluster_v2(v_lo + to, rank, lv);
      }
    }
    // Shared: every CTA's values are here after the barrier.  Otherwise it only keeps a CTA from
    // leaving while another reads its shared memory, and is waited for at the end.
    cluster_arrive();
    if (share) cluster_wait();
    late_wait = !share;
  }

  // ------------------------------------------------------------- out = y + v B^T
  // Warp: rows [16 wm, 16 wm + 16) and kCW columns of the chunk; v's fragments stay in registers
  // where they fit.  MMA column i of n8 tile 2a + b is column 16a + 4 (i / 2) + 2b + i % 2, so that
  // lane t ends with the four columns from 16a + 4t on and a quad stores whole 32-byte sectors.
  constexpr int WM = TM / 16, WN = kWarps / WM, kCW = kChunk / WN, kTiles = kCW / 8;
  constexpr bool kHold = RM <= 64;
  const int wm = warp % WM, wn = warp / WM;
  uint32_t vv[kHold ? RM / 16 : 1][2][4];
  const uint32_t vat = (uint32_t)((wm * 16 + (lmat & 1) * 8 + lrow) * S::BStride + (lmat >> 1) * 16);
  int orow[2];  // output rows of this lane's fragments
#pragma unroll
  for (int h = 0; h < 2; ++h) orow[h] = s_row[wm * 16 + h * 8 + g];
  int shift[2] = {0, 0};  // bytes by which their y lies behind the start of the chunk's rows
  if constexpr (kWindow) {
#pragma unroll
    for (int h = 0; h < 2; ++h) shift[h] = (int)(uintptr_t)(y + max(orow[h], 0) * L.ldy + c0) & 14;
  }
  for (int c = nk; c < chunks; ++c) {
    const uint32_t st = next();
    if (kHold && c == nk) {  // v is written by now for every thread
#pragma unroll
      for (int q = 0; q < RM / 16; ++q)
        if (q * 16 < R) {
          ldmatrix4(v_hi + vat + q * 32, vv[q][0]);
          ldmatrix4(v_lo + vat + q * 32, vv[q][1]);
        }
    }
    const int col = c0 + (c - nk) * kChunk + wn * kCW;
    if (col >= c1 || wm * 16 >= n) continue;
    float d[kTiles][4] = {};
#pragma unroll
    for (int q = 0; q < RM / 16; ++q) {
      if (q * 16 >= R) break;
      if (!kHold) {
        ldmatrix4(v_hi + vat + q * 32, vv[0][0]);
        ldmatrix4(v_lo + vat + q * 32, vv[0][1]);
      }
      const uint32_t (&v)[2][4] = vv[kHold ? q : 0];
      uint32_t bv[kTiles / 2][4];  // tile 2j (ranks low, high), tile 2j + 1
#pragma unroll
      for (int j = 0; j < kTiles / 2; ++j) {
        const int bc = wn * kCW + 16 * j + 4 * (lrow >> 1) + 2 * (lmat >> 1) + (lrow & 1);
        ldmatrix4(st + TM * kStride + bc * S::BStride + q * 32 + (lmat & 1) * 16, bv[j]);
      }
#pragma unroll
      for (int part = 0; part < 2; ++part)
#pragma unroll
        for (int j = 0; j < kTiles; ++j)
          mma_bf16(d[j], v[part], bv[j >> 1][2 * (j & 1)], bv[j >> 1][2 * (j & 1) + 1]);
    }
    const int left = c1 - (col + 4 * t);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (orow[h] < 0 || left <= 0) continue;
      const uint32_t from = st + (wm * 16 + h * 8 + g) * kStride + (wn * kCW + 4 * t) * 2 + shift[h];
      __nv_bfloat16* dst = reinterpret_cast<__nv_bfloat16*>(L.out) + orow[h] * L.ldo + col + 4 * t;
#pragma unroll
      for (int j = 0; j < kTiles; j += 2) {
        const uint2 w = kWindow ? ld_shared_4h(from + j * 16) : ld_shared_v2(from + j * 16);
        const __nv_bfloat162 lo = __floats2bfloat162_rn(__uint_as_float(w.x << 16) + d[j][2 * h],
                                                        __uint_as_float(w.x & 0xFFFF0000u) + d[j][2 * h + 1]);
        const __nv_bfloat162 hi = __floats2bfloat162_rn(__uint_as_float(w.y << 16) + d[j + 1][2 * h],
                                                        __uint_as_float(w.y & 0xFFFF0000u) + d[j + 1][2 * h + 1]);
        // without an adapter y's own bits (y + 0 would change -0 and NaNs)
        const uint32_t o[2] = {R ? *reinterpret_cast<const uint32_t*>(&lo) : w.x,
                               R ? *reinterpret_cast<const uint32_t*>(&hi) : w.y};
        if constexpr (VECY) {
          if (j * 8 < left) *reinterpret_cast<uint2*>(dst + j * 8) = make_uint2(o[0], o[1]);
        } else if (j * 8 + 4 <= left) {
          uint16_t* to = reinterpret_cast<uint16_t*>(dst + j * 8);
          if (!((uintptr_t)to & 7)) {
            *reinterpret_cast<uint2*>(to) = make_uint2(o[0], o[1]);
          } else if ((uintptr_t)to & 2) {
            to[0] = (uint16_t)o[0];
            *reinterpret_cast<uint32_t*>(to + 1) = __funnelshift_r(o[0], o[1], 16);
            to[3] = (uint16_t)(o[1] >> 16);
          } else {
            *reinterpret_cast<uint32_t*>(to) = o[0];
            *reinterpret_cast<uint32_t*>(to + 2) = o[1];
          }
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (j * 8 + i < left)
              reinterpret_cast<uint16_t*>(dst)[j * 8 + i] = (uint16_t)(o[i >> 1] >> ((i & 1) * 16));
        }
      }
    }
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  if (late_wait) cluster_wait();
}

template <int TM, int RM, int kCluster, bool VEC, bool VECY>
cudaError_t launch(const LoraLaunch& L, int64_t tiles, cudaStream_t s) {
  constexpr int bytes = LoraSmem<TM, RM, kCluster>::Bytes;
  static int done[64] = {0};
  const cudaError_t e = set_up_kernel(k_lora<TM, RM, kCluster, VEC, VECY>, bytes, done, kCluster > 8);
  if (e != cudaSuccess) return e;
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
  return cudaLaunchKernelEx(&cfg, k_lora<TM, RM, kCluster, VEC, VECY>, L);
}

template <int TM, int RM>
cudaError_t launch_vec(const LoraLaunch& L, cudaStream_t s) {
  // 16-byte copies need every row aligned and whole groups of 8
  const bool vec = ((uintptr_t)L.x | (uintptr_t)L.A | (uintptr_t)L.B) % 16 == 0 &&
                   (L.ldx | L.K | (int64_t)L.R) % 8 == 0;
  const bool vecy = ((uintptr_t)L.y | (uintptr_t)L.out) % 16 == 0 && (L.ldy | L.ldo | L.N) % 8 == 0;
  // at most one partial tile per group in use, the rows without adapter a group too
  const int64_t groups = L.M < L.L + 1 ? L.M : L.L + 1, tiles = groups + L.M / TM;
  if (!vec) return launch<TM, RM, 8, false, false>(L, tiles, s);
  // While clusters of 16 find an SM for each CTA, they halve what a CTA reads one after another
  // (1 row, 4096 -> 4096, rank 16: 5.1 us, 6.4 with 8, both with chunks of 128); beyond, 8 (96 rows
  // of 64 adapters, two CTAs per SM: 22.3 us, 30 with 16; 22.0 with 4, but then 1 row 9.5).
  if constexpr (TM == 16)
    if (tiles * 16 <= sm_count())
      return vecy ? launch<TM, RM, 16, true, true>(L, tiles, s) : launch<TM, RM, 16, true, false>(L, tiles, s);
  return vecy ? launch<TM, RM, 8, true, true>(L, tiles, s) : launch<TM, RM, 8, true, false>(L, tiles, s);
}

template <int RM>
cudaError_t launch_rank(const LoraLaunch& L, cudaStream_t s) {
  // Long runs of one adapter: tiles of 64 rows read the adapter a quarter as often.  4096 -> 4096,
  // rank 64, 4 adapters, 32 rows each: 9.6 us with 16 rows, 11.5 with 64; 96 rows: 14.7 and 13.8;
  // 5003 rows of 8 adapters, 4096 -> 5120, rank 32: 66 and 45.
  return L.M >= 64 * (int64_t)L.L ? launch_vec<64, RM>(L, s) : launch_vec<16, RM>(L, s);
}

}  // namespace

cudaError_t launch_lora(const LoraLaunch& L, cudaStream_t s) {
  if (L.R <= 32) return launch_rank<32>(L, s);
  if (L.R <= 64) return launch_rank<64>(L, s);
  return launch_rank<128>(L, s);
}

}  // namespace vt
