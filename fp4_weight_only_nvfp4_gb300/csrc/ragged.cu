// Products of ragged groups of rows: C[i] = A[row(i)] . W_e^T for the rows of every expert e in
// one call, with the packed FP4 weights dequantised inside.  Source: "dense projections take
// vLLM's own dense marlin" (vllm.cpp PR #54: the multi-expert route of the same W4A16 GEMM).
#include <cuda_bf16.h>

#include "common.cuh"
#include "handle.h"
#include "kernels.h"
#include "tc.cuh"

namespace vt {

namespace {

// Roles of one persistent CTA per SM (15 warps):
//   warp 0       weight producer: the packed 128 x 64 tiles of its items, one bulk copy per k step
//   warp 1       token producer: up to 256 rows x 64 k of bf16 activations per k step by tiled
//                TMA (128-byte swizzle), gathered four rows at a time where A is per token
//   warp 2       TMEM, and one thread issuing tcgen05.mma: D[128 weight rows][tokens] (fp32,
//                TMEM) += W . A^T with M = 128 and N = the tile's tokens rounded up to 16
//   warps 3-10   dequantisers: packed tile -> bf16 K-major swizzled MMA operand
//   warps 11-14  epilogue: lane = weight row, register = token
// The weights are the MMA's M operand so that its cost follows the tokens a group really has
// (N in steps of 16) and not a tile of 128 of them.  A weight value c * s (E2M1 times E4M3 or a
// power of two) has at most 6 significant bits: exact in bf16, so the activations go to the
// tensor core as they are, without a conversion pass.
// Items are (token tile, 128-row weight tile) pairs, weight tiles innermost; a group of n rows
// is cut into ceil(n / 256) token tiles of nearly equal size.
constexpr int kMaxTok = 256;
constexpr int kDeqWarps = 8;
constexpr int kThreads = (3 + kDeqWarps + 4) * 32;
constexpr int kNA = 3, kNB = 3, kNW = 13;    // ring depths: bf16 weights, tokens, packed weights
constexpr int kABytes = 128 * 128, kBBytes = kMaxTok * 128;
constexpr int kBoxRows = 16;                 // rows of one tiled activation load
constexpr uint64_t kWaitNs = 2000000000ull;
constexpr int kOffB = kNA * kABytes;
constexpr int kOffW = kOffB + kNB * kBBytes;
__host__ __device__ constexpr int off_x(int fmt) { return kOffW + kNW * tile_bytes(fmt); }
constexpr int kXBytes = 2 * 16 * 64 * 4;     // gate/up exchange of the SiLU epilogue
constexpr int kNumBars = 2 * (kNA + kNB + kNW) + 4 + 1;
__host__ __device__ constexpr int off_bar(int fmt) { return off_x(fmt) + kXBytes; }
__host__ __device__ constexpr int off_tab(int fmt) { return off_bar(fmt) + (kNumBars + 1) * 8; }
// prefix sums of the groups' token tiles, and their first rows
inline int ragged_smem(int fmt, int E) { return off_tab(fmt) + 2 * (E + 1) * 4 + 1024; }

constexpr uint32_t kIdescBase = (1u << 4) | (1u << 7) | (1u << 10) | ((128u >> 4) << 24);

__device__ __forceinline__ float silu_f(float x) { return x / (1.0f + expf(-x)); }

__device__ __forceinline__ __nv_bfloat162 as_bf162(uint32_t x) {
  return *reinterpret_cast<__nv_bfloat162*>(&x);
}
__device__ __forceinline__ uint32_t as_u32(__nv_bfloat162 x) {
  return *reinterpret_cast<uint32_t*>(&x);
}

// f16x2 of two E2M1 values c -> bf16x2 of c * 2^-112: the sign stays, exponent and mantissa move
// down by the 3 bits that the mantissas differ in (an E2M1 value's low 9 mantissa bits are 0, so
// nothing crosses into the lower half).
__device__ __forceinline__ uint32_t f16x2_to_bf16x2_m112(uint32_t h) {
  return ((h >> 3) & 0x0FFF0FFFu) | (h & 0x80008000u);
}

struct Item {
  int e, rt, n;     // group, weight row tile, tokens
  int64_t i0;       // first grouped row
};

// The item's group by bisection of the token tiles' prefix sums.
__device__ __forceinline__ Item item_at(int64_t it, const RaggedLaunch& L, const int* tstart,
                                        const int* first) {
  Item q;
  const int tile = (int)(it / L.RT);
  q.rt = (int)(it - (int64_t)tile * L.RT);
  int lo = 0, hi = L.E;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (tstart[mid] <= tile) lo = mid;
    else hi = mid;
  }
  q.e = lo;
  const int nt = tstart[lo + 1] - tstart[lo], t = tile - tstart[lo];
  const int64_t n = first[lo + 1] - first[lo];
  const int64_t b = n * t / nt;
  q.n = (int)(n * (t + 1) / nt - b);
  q.i0 = first[lo] + b;
  return q;
}

template <int FMT, bool GATHER, bool SILU>
__global__ void __launch_bounds__(kThreads, 1)
    k_ragged(const __grid_constant__ CUtensorMap tmA, const RaggedLaunch L) {
  constexpr int TB = tile_bytes(FMT);
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_u = smem_u32(smem_raw);
  const uint32_t base_u = (raw_u + 1023u) & ~1023u;
  uint8_t* base = smem_raw + (base_u - raw_u);
  const uint32_t sA = base_u, sB = base_u + kOffB, sW = base_u + kOffW;
  float* s_x = reinterpret_cast<float*>(base + off_x(FMT));
  const uint32_t bars = base_u + off_bar(FMT);
  const uint32_t a_full = bars, a_empty = a_full + 8 * kNA;
  const uint32_t b_full = a_empty + 8 * kNA, b_empty = b_full + 8 * kNB;
  const uint32_t w_full = b_empty + 8 * kNB, w_empty = w_full + 8 * kNW;
  const uint32_t acc_full = w_empty + 8 * kNW, acc_empty = acc_full + 16, drain = acc_empty + 16;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(base + off_bar(FMT) + kNumBars * 8);
  volatile int* abort = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* tstart = reinterpret_cast<int*>(base + off_tab(FMT));
  int* first = tstart + L.E + 1;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kNA; ++s) {
      mbar_init(a_full + 8 * s, kDeqWarps);
      mbar_init(a_empty + 8 * s, 1);
    }
    for (int s = 0; s < kNB; ++s) {
      mbar_init(b_full + 8 * s, 1);
      mbar_init(b_empty + 8 * s, 1);
    }
    for (int s = 0; s < kNW; ++s) {
      mbar_init(w_full + 8 * s, 1);
      mbar_init(w_empty + 8 * s, kDeqWarps);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(acc_full + 8 * s, 1);
      mbar_init(acc_empty + 8 * s, 4);
    }
    mbar_init(drain, 1);
    *abort = 0;
  }
  if (warp == 2) tmem_alloc(smem_u32(tmem_slot), 512);
  fence_mbar_init();
  // everything above needs nothing of the kernel before this one
  pdl_wait();
  pdl_launch_dependents();
  bool bad = false;  // offsets out of order or out of range
  for (int e = threadIdx.x; e <= L.E; e += kThreads) {
    const int64_t v = L.offsets[e], c = v < 0 ? 0 : (v > L.pairs ? L.pairs : v);
    bad |= v != c;
    first[e] = (int)c;
  }
  __syncthreads();
  if (warp == 0) {  // token tiles of each group, summed up
    const int per = (L.E + 31) / 32;
    int sum = 0;
    for (int e = lane * per; e < (lane + 1) * per && e < L.E; ++e) {
      const int n = first[e + 1] - first[e];
      bad |= n < 0;
      sum += n > 0 ? (n + kMaxTok - 1) / kMaxTok : 0;
    }
    int run = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, run, o);
      if (lane >= o) run += u;
    }
    run -= sum;
    for (int e = lane * per; e < (lane + 1) * per && e < L.E; ++e) {
      tstart[e] = run;
      const int n = first[e + 1] - first[e];
      run += n > 0 ? (n + kMaxTok - 1) / kMaxTok : 0;
    }
    if (lane == 31) tstart[L.E] = run;
    if (blockIdx.x == 0 && bad) atomicExch(L.status, 6);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int64_t items = (int64_t)tstart[L.E] * L.RT, G = gridDim.x;
  const int KT = (int)L.KT;

  if (warp == 0) {
    // ---------------------------------------------------------- weight producer
    if (lane == 0) {
      const uint64_t pol = l2_evict_normal_policy();
      uint32_t iw = 0, pw = 0;
      int issued = 0;
      bool ok = true;
      for (int64_t it = blockIdx.x; ok && it < items; it += G) {
        const Item q = item_at(it, L, tstart, first);
        const uint8_t* src = reinterpret_cast<const uint8_t*>(L.packed) + q.e * L.expert_bytes +
                             kHeaderBytes + (int64_t)q.rt * KT * TB;
        for (int kt = 0; kt < KT; ++kt) {
          if (!(ok = pf_wait(w_empty + 8 * iw, pw ^ 1u, abort, kWaitNs))) break;
          mbar_expect_tx(w_full + 8 * iw, TB);
          bulk_g2s(sW + iw * TB, src + (int64_t)kt * TB, TB, w_full + 8 * iw, pol);
          ++issued;
          if (++iw == kNW) { iw = 0; pw ^= 1u; }
        }
      }
      if (!ok) {  // let the copies in flight land before shared memory is released
        atomicExch(L.status, 5);
        for (int k = 0; k < kNW && k < issued; ++k) {
          iw = iw == 0 ? kNW - 1 : iw - 1;
          if (iw == kNW - 1) pw ^= 1u;
          const uint64_t t0 = globaltimer_ns();
          while (!mbar_try_wait(w_full + 8 * iw, pw) && globaltimer_ns() - t0 < kWaitNs) {}
        }
      }
    }
  } else if (warp == 1) {
    // ----------------------------------------------------------- token producer
    const uint64_t pol = l2_evict_last_policy();
    uint32_t ib = 0, pb = 0;
    int issued = 0;
    bool ok = true;
    for (int64_t it = blockIdx.x; ok && it < items; it += G) {
      const Item q = item_at(it, L, tstart, first);
      const int n16 = (q.n + 15) & ~15;
      // gathered: lane l fetches rows 4l .. 4l+3 and 128 + 4l ..; past the tile's tokens the
      // last one again (its products are not stored)
      int4 y[2];
      if constexpr (GATHER) {
        for (int h = 0; h < 2; ++h) {
          int r[4];
          for (int c = 0; c < 4; ++c) {
            const int i = h * 128 + lane * 4 + c;
            const int p = __ldg(L.order + q.i0 + (i < q.n ? i : q.n - 1));
            const bool in = p >= 0 && p < L.pairs;
            if (!in) atomicExch(L.status, 6);
            r[c] = in ? p / L.topk : 0;
          }
          y[h] = make_int4(r[0], r[1], r[2], r[3]);
        }
      }
      for (int kt = 0; kt < KT; ++kt) {
        ok = lane != 0 || pf_wait(b_empty + 8 * ib, pb ^ 1u, abort, kWaitNs);
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (!ok) break;
        const uint32_t dst = sB + ib * kBBytes, bar = b_full + 8 * ib;
        if (lane == 0) mbar_expect_tx(bar, (uint32_t)n16 * 128u);
        __syncwarp();
        if constexpr (GATHER) {
          if (lane * 4 < n16) tma_gather4(dst + lane * 512, &tmA, kt * kTileK, y[0], bar, pol);
          if (128 + lane * 4 < n16)
            tma_gather4(dst + 16384 + lane * 512, &tmA, kt * kTileK, y[1], bar, pol);
        } else {
          if (lane * kBoxRows < n16)
            tma_load_2d(dst + lane * kBoxRows * 128, &tmA, kt * kTileK, (int)q.i0 + lane * kBoxRows,
                        bar, pol);
        }
        ++issued;
        if (++ib == kNB) { ib = 0; pb ^= 1u; }
      }
    }
    if (!ok && lane == 0) {
      atomicExch(L.status, 5);
      for (int k = 0; k < kNB && k < issued; ++k) {
        ib = ib == 0 ? kNB - 1 : ib - 1;
        if (ib == kNB - 1) pb ^= 1u;
        const uint64_t t0 = globaltimer_ns();
        while (!mbar_try_wait(b_full + 8 * ib, pb) && globaltimer_ns() - t0 < kWaitNs) {}
      }
    }
    __syncwarp();
  } else if (warp == 2) {
    // --------------------------------------------------------------- MMA issuer
    if (lane == 0) {
      uint32_t ia = 0, pa = 0, ib = 0, pb = 0, ic = 0, pc = 0;
      bool ok = true;
      for (int64_t it = blockIdx.x; ok && it < items; it += G) {
        const Item q = item_at(it, L, tstart, first);
        const uint32_t idesc = kIdescBase | ((uint32_t)((q.n + 15) >> 4) << 18);
        const uint32_t d = tmem + ic * kMaxTok;
        if (!(ok = pf_wait(acc_empty + 8 * ic, pc ^ 1u, abort, kWaitNs))) break;
        tc_fence_after();
        for (int kt = 0; kt < KT; ++kt) {
          if (!(ok = pf_wait(b_full + 8 * ib, pb, abort, kWaitNs))) break;
          if (!(ok = pf_wait(a_full + 8 * ia, pa, abort, kWaitNs))) break;
          tc_fence_after();
          const uint64_t ad = desc_sw128(sA + ia * kABytes), bd = desc_sw128(sB + ib * kBBytes);
#pragma unroll
          for (int kk = 0; kk < kTileK / 16; ++kk)  // +32 bytes per 16-element k step
            mma_f16(d, ad + 2 * kk, bd + 2 * kk, idesc, (kt > 0 || kk > 0) ? 1u : 0u);
          mma_commit(a_empty + 8 * ia);
          mma_commit(b_empty + 8 * ib);
          if (++ia == kNA) { ia = 0; pa ^= 1u; }
          if (++ib == kNB) { ib = 0; pb ^= 1u; }
        }
        if (!ok) break;
        mma_commit(acc_full + 8 * ic);
        if (++ic == 2) { ic = 0; pc ^= 1u; }
      }
      if (!ok) atomicExch(L.status, 5);
      mma_commit(drain);  // every MMA issued has completed once this commit arrives
      const uint64_t t0 = globaltimer_ns();
      while (!mbar_try_wait(drain, 0) && globaltimer_ns() - t0 < kWaitNs) {}
    }
  } else if (warp < 3 + kDeqWarps) {
    // ------------------------------------------------------------- dequantisers
    // Warp d owns row block d: lane (g, t) holds rows 16d + g and 16d + g + 8 for physical k
    // [16t, 16t + 16) of the k tile (one NVFP4 scale each).
    const int d = warp - 3, g = lane >> 2, t = lane & 3;
    const int soff = scale_offset(FMT, d, g, t);
    const int row = 16 * d + g;  // row & 7 == (row + 8) & 7 == g
    const uint32_t c0 = (uint32_t)(((2 * t) ^ g) << 4), c1 = (uint32_t)(((2 * t + 1) ^ g) << 4);
    uint32_t iw = 0, pw = 0, ia = 0, pa = 0;
    bool ok = true;
    for (int64_t it = blockIdx.x; ok && it < items; it += G) {
      bool wide = false;
      if constexpr (FMT == FMT_MX) {
        const Item q = item_at(it, L, tstart, first);
        wide = reinterpret_cast<const PackedHeader*>(reinterpret_cast<const uint8_t*>(L.packed) +
                                                     q.e * L.expert_bytes)->wide != 0;
      }
      for (int kt = 0; kt < KT; ++kt) {
        if (!(ok = pf_wait(w_full + 8 * iw, pw, abort, kWaitNs))) break;
        const uint32_t tb = sW + iw * TB;
        const int4 cw = ld_shared_v4(tb + d * 512 + lane * 16);
        const uint32_t sc = ld_shared_u16(tb + soff);
        const uint32_t words[4] = {(uint32_t)cw.x, (uint32_t)cw.y, (uint32_t)cw.z, (uint32_t)cw.w};
        uint32_t og[8], o8[8];  // rows g and g + 8, k order, bf16x2
        if (FMT == FMT_MX && wide) {
          // raw E8M0 bytes: c * 2^(e - 127) by fp32, exact in bf16 (subnormals included)
          const float wg = e8m0_to_f32(sc & 0xFFu), w8 = e8m0_to_f32((sc >> 8) & 0xFFu);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            uint32_t c4[4], o4[4];
            e2m1x8_to_f16x8(words[q], c4[0], c4[1], c4[2], c4[3]);
#pragma unroll
            for (int b = 0; b < 4; ++b) {
              const __half2 hc = *reinterpret_cast<const __half2*>(&c4[b]);
              const float s = (b & 1) ? w8 : wg;
              o4[b] = as_u32(__floats2bfloat162_rn(__low2float(hc) * s, __high2float(hc) * s));
            }
            og[2 * q] = o4[0];
            og[2 * q + 1] = o4[2];
            o8[2 * q] = o4[1];
            o8[2 * q + 1] = o4[3];
          }
        } else {
          const uint32_t s2 = FMT == FMT_NV ? e4m3x2_to_f16x2(sc) : mxenc2_to_f16x2(sc);
          const __half2 sh = *reinterpret_cast<const __half2*>(&s2);
          const float fg = __low2float(sh) * 0x1p112f, f8 = __high2float(sh) * 0x1p112f;
          const __nv_bfloat162 bg = __floats2bfloat162_rn(fg, fg), b8 = __floats2bfloat162_rn(f8, f8);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            uint32_t r0, r1, r2, r3;
            e2m1x8_to_f16x8(words[q], r0, r1, r2, r3);
            og[2 * q] = as_u32(__hmul2(as_bf162(f16x2_to_bf16x2_m112(r0)), bg));
            o8[2 * q] = as_u32(__hmul2(as_bf162(f16x2_to_bf16x2_m112(r1)), b8));
            og[2 * q + 1] = as_u32(__hmul2(as_bf162(f16x2_to_bf16x2_m112(r2)), bg));
            o8[2 * q + 1] = as_u32(__hmul2(as_bf162(f16x2_to_bf16x2_m112(r3)), b8));
          }
        }
        // every lane has used what it loaded: only now may the next copy overwrite the stage
        __syncwarp();
        if (lane == 0) mbar_arrive(w_empty + 8 * iw);
        if (++iw == kNW) { iw = 0; pw ^= 1u; }
        if (!(ok = pf_wait(a_empty + 8 * ia, pa ^ 1u, abort, kWaitNs))) break;
        const uint32_t rg = sA + ia * kABytes + row * 128, r8 = rg + 8 * 128;
        st_shared_v4(rg + c0, og[0], og[1], og[2], og[3]);
        st_shared_v4(rg + c1, og[4], og[5], og[6], og[7]);
        st_shared_v4(r8 + c0, o8[0], o8[1], o8[2], o8[3]);
        st_shared_v4(r8 + c1, o8[4], o8[5], o8[6], o8[7]);
        fence_proxy_async_smem();  // generic-proxy writes -> visible to the tensor core
        __syncwarp();
        if (lane == 0) mbar_arrive(a_full + 8 * ia);
        if (++ia == kNA) { ia = 0; pa ^= 1u; }
      }
    }
    if (!ok && lane == 0) atomicExch(L.status, 5);
  } else {
    // ----------------------------------------------------------------- epilogue
    const int qd = warp & 3;  // TMEM lane quarter this warp may access
    const int r = qd * 32 + lane;  // packed row of the tile
    __nv_bfloat16* C = reinterpret_cast<__nv_bfloat16*>(L.C);
    uint32_t ic = 0, pc = 0;
    bool ok = true;
    for (int64_t it = blockIdx.x; ok && it < items; it += G) {
      const Item q = item_at(it, L, tstart, first);
      const PackedHeader* hdr = reinterpret_cast<const PackedHeader*>(
          reinterpret_cast<const uint8_t*>(L.packed) + q.e * L.expert_bytes);
      if (!(ok = pf_wait(acc_full + 8 * ic, pc, abort, kWaitNs))) break;
      tc_fence_after();
      const uint32_t ta = tmem + ic * kMaxTok + ((uint32_t)(qd * 32) << 16);
      if constexpr (SILU) {
        // lanes 0-63 hold gate rows, 64-127 the matching up rows: for every 32 tokens the gate
        // warps finish the first 16 and the up warps the others, trading the halves they lack
        const float f = hdr->factor[qd >> 1];
        const int64_t col = (int64_t)q.rt * 64 + (r & 63);
        const bool live = col < L.seg_split, up = qd >= 2;
        for (int c = 0; c * 32 < q.n; ++c) {
          uint32_t v[32];
          tmem_ld32(ta + c * 32, v);
          const int64_t i = q.i0 + c * 32 + lane;
          int64_t out = i;
          if (L.scatter && c * 32 + lane < q.n) out = L.order[i];
          asm volatile("bar.sync 1, 128;" ::: "memory");  // the halves of the chunk before are read
          float* mine = s_x + (up ? 0 : 16 * 64);
#pragma unroll
          for (int j = 0; j < 16; ++j)
            mine[j * 64 + (r & 63)] = __uint_as_float(up ? v[j] : v[16 + j]) * f;
          asm volatile("bar.sync 1, 128;" ::: "memory");
          const float* other = s_x + (up ? 16 * 64 : 0);
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const int tok = c * 32 + (up ? 16 : 0) + j;
            const int64_t ro = __shfl_sync(0xffffffffu, out, (up ? 16 : 0) + j);
            const float x = __uint_as_float(up ? v[16 + j] : v[j]) * f;
            const float z = other[j * 64 + (r & 63)];
            const float h = up ? silu_f(z) * x : silu_f(x) * z;
            if (tok < q.n && live && ro >= 0 && ro < L.pairs)
              C[ro * L.ldc + col] = __float2bfloat16_rn(h);
          }
        }
      } else {
        const int64_t n = packed_to_row(L.layout, (int64_t)q.rt * kTileRows + r, L.N, L.seg_split);
        const float f = hdr->factor[n >= L.seg_split ? 1 : 0];
        for (int c = 0; c * 32 < q.n; ++c) {
          uint32_t v[32];
          tmem_ld32(ta + c * 32, v);
          const int64_t i = q.i0 + c * 32 + lane;
          int64_t out = i;
          if (L.scatter && c * 32 + lane < q.n) {
            out = L.order[i];
            if ((out < 0 || out >= L.pairs) && q.rt == 0) atomicExch(L.status, 6);
          }
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            const int64_t ro = __shfl_sync(0xffffffffu, out, j);
            if (c * 32 + j < q.n && n >= 0 && ro >= 0 && ro < L.pairs)
              C[ro * L.ldc + n] = __float2bfloat16_rn(__uint_as_float(v[j]) * f);
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(acc_empty + 8 * ic);
      if (++ic == 2) { ic = 0; pc ^= 1u; }
    }
    if (!ok && lane == 0) atomicExch(L.status, 5);
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
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

namespace {

template <int FMT, bool GATHER, bool SILU>
cudaError_t launch_main(const CUtensorMap& tm, const RaggedLaunch& L, int grid, cudaStream_t s) {
  static int done[64] = {0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!done[dev]) {
    e = cudaFuncSetAttribute(k_ragged<FMT, GATHER, SILU>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             ragged_smem(FMT, kMaxGroups));
    if (e != cudaSuccess) return e;
    done[dev] = 1;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = (size_t)ragged_smem(FMT, L.E);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_ragged<FMT, GATHER, SILU>, tm, L);
}

template <int FMT>
cudaError_t launch_fmt(const CUtensorMap& tm, const RaggedLaunch& L, int grid, cudaStream_t s) {
  if (L.gather) return L.silu ? launch_main<FMT, true, true>(tm, L, grid, s)
                              : launch_main<FMT, true, false>(tm, L, grid, s);
  return L.silu ? launch_main<FMT, false, true>(tm, L, grid, s)
                : launch_main<FMT, false, false>(tm, L, grid, s);
}

}  // namespace

cudaError_t launch_ragged(const RaggedLaunch& L, cudaStream_t s) {
  auto enc = tensor_map_encoder();
  if (!enc) return cudaErrorNotSupported;
  // A as a 2-D tensor {K, rows}: reads past K or past the last row return zeros
  CUtensorMap tm;
  const int64_t rows = L.gather ? L.pairs / L.topk : L.pairs;
  const cuuint64_t dims[2] = {(cuuint64_t)L.K, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)L.lda * 2};
  const cuuint32_t box[2] = {(cuuint32_t)kTileK, (cuuint32_t)(L.gather ? 1 : kBoxRows)};
  const cuuint32_t estr[2] = {1, 1};
  if (enc(&tm, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(L.A), dims, strides, box, estr,
          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
          CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return cudaErrorInvalidValue;
  // at most one partial token tile per group in use
  const int64_t groups = L.pairs < L.E ? L.pairs : L.E;
  const int64_t most = (groups + L.pairs / kMaxTok) * L.RT;
  int64_t grid = sm_count();
  if (grid > most) grid = most;
  return L.fmt == FMT_NV ? launch_fmt<FMT_NV>(tm, L, (int)grid, s)
                         : launch_fmt<FMT_MX>(tm, L, (int)grid, s);
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
