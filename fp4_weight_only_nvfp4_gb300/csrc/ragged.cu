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

// Operands: f16.  A pre-pass writes the activations as A * 2^-p (one power of two per row), and a
// weight value c * s (at most 6 significant bits) is exact in f16, one multiply away from the
// E2M1 conversion.  An expert whose E8M0 scales span more exponents than f16 holds (`wide`) takes
// bf16, in which its values and the caller's activations are exact.
//
// Roles of one persistent CTA per SM (28 warps):
//   warp 0       weight producer: R packed 128 x 64 tiles (one bulk copy each) per k step
//   warp 1       token producer: up to TOK rows x 64 k of activations per k step by tiled TMA
//                (128-byte swizzle), where the pre-pass has put the rows in group order
//   warps 2, 3   one thread each issuing tcgen05.mma for row tile 0 and 1: D[128 weight rows]
//                [tokens] (fp32, TMEM) += W . A^T, M = 128 and N = the tile's tokens rounded up to
//                16 (one thread for both took 700 cycles per k step to issue 256 cycles of MMAs)
//   Sets x 4     dequantisers: packed tiles -> 16-bit MMA operand in TMEM; a set of four warps
//   warps        takes every Sets-th k step, each warp its TMEM quarter (32 rows) of each tile
//   4 warps      (LOAD) loaders: gathered rows by asynchronous copies to the token stage
//   last 8 warps epilogue
// The weights are the MMA's M operand so that its cost follows the tokens a group really has
// (N in steps of 16), and they go to the tensor core through TMEM: a weight tile in shared memory
// would be written and read once per token tile, which alone took twice the time that its packed
// form takes to arrive from HBM (77 tokens x top-8 over 128 experts of 1536 x 2048: 61 us; 47).
// Token tiles: an M = 128, K = 16 MMA takes N / 2 cycles and some 27 more (58 measured at N = 64, 89
// at 128), and no less than 60 to 70 where N is small, so
//   TOK = 64  for few rows per group, where that time hides behind the weights' arrival: two
//             accumulators per row tile, the epilogue of an item beside the MMAs of the next;
//   TOK = 128 for many: the accumulators of one item and the weight stages fill TMEM, so the
//             epilogue first moves an item to shared memory as bf16 and then stores it.  (160 rows
//             leave room for three stages only, which cost 8 % at 4096 tokens of top-8.)
// Bound: with few rows per group by that least time of an MMA, 270 cycles per packed tile of 4.6 KB
// or 5.3 TB/s over 152 SMs (77 tokens: 43 us, 5.3 TB/s of packed weights); with many by the MMAs and
// by the drains, in which an item's SiLU (two special-function operations per output) holds up the
// next item's MMAs for 2000 of its 20000 cycles (4096 tokens: 155 us, 1.33 PFLOP/s, of a call's 166).
// With SiLU and two row tiles the dequantisers put the gate rows of both tiles in accumulator 0
// and the up rows in accumulator 1, so that a thread finds its pairs in the same lane.
// Items are (token tile, R x 128 weight rows) pairs, weight rows innermost; a group of n rows is
// cut into ceil(n / TOK) token tiles of nearly equal size.
//
// k order: a dequantiser's lane (g, t) holds 16 consecutive k of its rows, and the TMEM store that
// takes them there gives it, of every 8 columns (k pairs), columns 2t and 2t + 1.  So pair
// 8t + 2q + i of a 64-k tile is the MMA's pair 8q + 2t + i, and the activations are laid out in
// that order (by the pre-pass).
constexpr int kThreads = 28 * 32;
constexpr int kDeqWarp0 = 4;                 // first of the dequantisers
constexpr int kEpiWarp0 = 20;                // first of the epilogue warps
constexpr int kNS = 4;                       // stages of dequantised weights (TMEM) and tokens
constexpr int kTileTable = 1024;             // token tiles whose group is looked up, not searched
constexpr uint64_t kWaitNs = 2000000000ull;   // limit of a wait (of the roles: unless the call sets one)
constexpr int kNoHold = 1 << 30;
constexpr uint64_t kPauseNs = 1000000ull;     // of a producer that is asked to pause

// Shared-memory map (from a 1024-byte aligned base).
template <int FMT, int R, bool LOAD, int TOK>
struct Map {
  static constexpr int BBytes = TOK * 128;
  static constexpr int Box = TOK / 4;              // rows of one tiled activation load
  static constexpr int Sets = LOAD ? 3 : 4;        // sets of dequantisers
  static constexpr int NW = R == 1 ? 16 : TOK == 64 ? 14 : 8;  // stages of packed weights
  // A wait on a phase's parity holds only if the phase before it is known to be over.  A set
  // that waits for k step c has passed its wait of step c - Sets for a free stage, so the steps
  // up to c - Sets - NS have been multiplied; the steps that used the same stage and the same
  // packed stage before, c - NS and c - NW, have their phases before last over (Sets <= NS) and
  // last over (the packed copies land in any order, so nothing less than consumption tells).
  static_assert(Sets <= kNS && NW >= kNS + Sets, "barrier phases");
  static constexpr int OffW = kNS * BBytes;
  static constexpr int OffX = OffW + NW * R * tile_bytes(FMT);
  // epilogue.  R = 2: an item's TOK x 256 outputs in bf16, token rows 16 bytes apart (SiLU: x
  // 128).  R = 1, per group of four warps: 2 x 16 tokens x 128 columns; with SiLU 2 x 16 x 64
  // behind the exchange of 2 x 4 warps x 8 registers.
  static constexpr int XGroup = 8192 + 2 * 16 * 144;
  static constexpr int XBytes = R == 2 ? TOK * 528 : 2 * XGroup;
  static constexpr int OffTok = OffX + XBytes;     // 2 (R = 1: per group) x TOK x {output row, scale}
  static constexpr int OffBar = OffTok + 2 * (R == 2 ? 1 : 2) * TOK * 8;
  static constexpr int NumBars = 2 * (kNS + NW) + 4 + 2;
  static constexpr int OffTab = OffBar + (NumBars + 2) * 8;  // behind TMEM's address, abort and issued
  // per group: prefix sum of the token tiles, first row, rows per tile; group of a token tile
  static constexpr int smem(int E) { return OffTab + (E + 1) * 10 + kTileTable * 2 + 16 + 1024; }
  static_assert(2 * 16 * 272 <= XGroup, "plain epilogue");
  static_assert(OffTab + (kMaxGroups + 1) * 10 + kTileTable * 2 + 16 + 1024 <= 227 * 1024, "shared memory");
};

// TMEM columns: accumulators [Bufs][R][TOK] of fp32, then the weight stages [kNS][R][32] of pairs.
template <int R, int TOK>
struct Tmem {
  static constexpr uint32_t Bufs = TOK == 64 ? 2 : 1;
  static constexpr uint32_t A = Bufs * R * TOK, Cols = A + kNS * R * 32;
  static_assert(Cols == 256 || Cols == 512, "a power of two");
};

constexpr uint32_t kIdescF16 = (1u << 4) | ((128u >> 4) << 24);
constexpr uint32_t kIdescBF16 = kIdescF16 | (1u << 7) | (1u << 10);

struct RaggedParams {
  RaggedLaunch L;
  const __half* Ap;       // converted activations [rows][ldp], in group order; LOAD: per token
  int64_t ldp;
  const float* rowscale;  // 2^p of each of their rows
  uint64_t wait_ns;       // limit of the roles' waits
  int hold;               // k steps after which each weight producer stops, or pauses
};

// SiLU(x) = x / (1 + e^-x) by the hardware's 2^x and 1/x (each good to 2^-22; the product before
// 2^x adds |x| 2^-24): far inside the rounding of the result to bf16.  From 1 + e^-x > 2^126 on
// the reciprocal is 0, for a value below 2^-119.  With expf and a division the epilogue of 4096
// tokens held up the MMAs for a sixth of the time.
__device__ __forceinline__ float silu_f(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + __expf(-x)));
  return x * r;
}

__device__ __forceinline__ uint32_t as_u32(__nv_bfloat162 x) {
  return *reinterpret_cast<uint32_t*>(&x);
}

// 16 TMEM lanes x 16 columns of fp32 as MMA fragments: with lane = 4g + t, v[0..1] are row g,
// columns 2t and 2t + 1, v[2..3] row g + 8, v[4..7] the same 8 columns on.
__device__ __forceinline__ void tmem_ld_frag(uint32_t taddr, uint32_t (&v)[8]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]),
        "=r"(v[7])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_wait_frags(uint32_t (&a)[8], uint32_t (&b)[8]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(a[0]), "+r"(a[1]), "+r"(a[2]), "+r"(a[3]), "+r"(a[4]), "+r"(a[5]),
                 "+r"(a[6]), "+r"(a[7]), "+r"(b[0]), "+r"(b[1]), "+r"(b[2]), "+r"(b[3]),
                 "+r"(b[4]), "+r"(b[5]), "+r"(b[6]), "+r"(b[7])
               :
               : "memory");
}
// Four 8 x 8 matrices of 16-bit values, transposed, to the rows whose addresses the lanes give.
__device__ __forceinline__ void stmatrix_t4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c,
                                            uint32_t d) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr),
               "r"(a), "r"(b), "r"(c), "r"(d)
               : "memory");
}
// 16 bytes global -> shared, asynchronous.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// 8 bytes; zeros where `bytes` is 0.
__device__ __forceinline__ void cp_async8(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ bool mbar_test_wait(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n"
      " selp.u32 %0, 1, 0, p;\n}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
// Bounded wait that also gives up when another role has.  The thread sleeps on the barrier for up
// to 0.1 ms at a time: two dozen warps asking again and again slowed the others' barrier
// operations (77 tokens x top-8 over 128 experts: 48 -> 43 us).  Each thread gets an answer of its
// own: with the limit running out while the barrier completes, one thread may be told to give up
// and its neighbour to go on.  Whoever shares a warp-wide instruction or a named barrier first agrees
// on one answer (warp_wait, team_wait).
__device__ __forceinline__ bool mbar_sleep_wait(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, 100000;\n"
      " selp.u32 %0, 1, 0, p;\n}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ bool stage_wait(uint32_t bar, uint32_t parity, volatile int* abort,
                                           const RaggedParams& p) {
  if (mbar_sleep_wait(bar, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
  while (true) {
    if (*abort) return false;
    if (mbar_sleep_wait(bar, parity)) return true;
    if (globaltimer_ns() - t0 > p.wait_ns) {
      *abort = 1;
      return false;
    }
  }
}
// stage_wait with one answer for the warp: false if it is for any lane.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int* abort,
                                          const RaggedParams& p) {
  return __all_sync(0xffffffffu, stage_wait(bar, parity, abort, p));
}
// stage_wait with one answer for the `Threads` threads of named barrier `id`, which also
// synchronises them: a thread that gives up still arrives, so none is waited for in vain.
template <int Threads>
__device__ __forceinline__ bool team_wait(int id, uint32_t bar, uint32_t parity, volatile int* abort,
                                          const RaggedParams& p) {
  const uint32_t mine = stage_wait(bar, parity, abort, p) ? 1u : 0u;
  uint32_t all;
  __syncwarp();
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.b32 p, %1, 0;\n bar.red.and.pred q, %2, %3, p;\n"
      " selp.u32 %0, 1, 0, q;\n}"
      : "=r"(all)
      : "r"(mine), "r"(id), "n"(Threads)
      : "memory");
  return all != 0;
}
// D[tmem] (+)= A[tmem] . B[smem desc]^T, kind::f16, one thread.
__device__ __forceinline__ void mma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                           uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// 16 lanes x 32 columns to TMEM in the layout of tmem_ld_frag (four times 8 columns): of columns
// 8q .. 8q + 7 this lane gives 2t, 2t + 1 of row g (lo) and of row g + 8 (hi).
__device__ __forceinline__ void tmem_st_frag(uint32_t taddr, const uint32_t (&lo)[8],
                                             const uint32_t (&hi)[8]) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x256b.x4.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
      "%12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(lo[0]), "r"(lo[1]), "r"(hi[0]), "r"(hi[1]), "r"(lo[2]), "r"(lo[3]), "r"(hi[2]), "r"(hi[3]),
      "r"(lo[4]), "r"(lo[5]), "r"(hi[4]), "r"(hi[5]), "r"(lo[6]), "r"(lo[7]), "r"(hi[6]), "r"(hi[7])
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
// The byte in a 128-byte row of the first of the two MMA pairs that physical k pairs 4c + 2j and
// 4c + 2j + 1 (16-byte chunk c, half j) become.
__device__ __forceinline__ uint32_t pair_byte(int c, int j) {
  return (uint32_t)(32 * (2 * (c & 1) + j) + 8 * (c >> 1));
}
// Arrives on `bar` once this thread's copies so far have landed.
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  return as_u32(__floats2bfloat162_rn(a, b));
}

// The groups' token tiles, in shared memory.
struct Tiles {
  int* start;      // [E + 1] prefix sums of the token tiles
  int* first;      // [E + 1] first grouped row
  uint16_t* rows;  // [E] rows per token tile
  uint16_t* of;    // [kTileTable] group of a token tile
  int E;
};

struct Item {
  int e, n;      // group, tokens
  int64_t i0;    // first grouped row
};

__device__ __forceinline__ Item item_of(const Tiles& T, int tile) {
  Item q;
  if (tile < kTileTable) {
    q.e = T.of[tile];
  } else {
    int lo = 0, hi = T.E;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (T.start[mid] <= tile) lo = mid;
      else hi = mid;
    }
    q.e = lo;
  }
  const int per = T.rows[q.e], b = (tile - T.start[q.e]) * per;
  const int left = T.first[q.e + 1] - T.first[q.e] - b;
  q.n = left < per ? left : per;
  q.i0 = T.first[q.e] + b;
  return q;
}

// A CTA's walk over its items: (token tile, group of R row tiles), G items apart.
struct Walk {
  int tile, rg, dtile, drg, RG;
  __device__ __forceinline__ Walk(int64_t RGs) {
    RG = (int)RGs;
    tile = (int)blockIdx.x / RG;
    rg = (int)blockIdx.x - tile * RG;
    dtile = (int)gridDim.x / RG;
    drg = (int)gridDim.x - dtile * RG;
  }
  __device__ __forceinline__ void next() {
    tile += dtile;
    if ((rg += drg) >= RG) {
      rg -= RG;
      ++tile;
    }
  }
};

__device__ __forceinline__ const PackedHeader* header_of(const RaggedLaunch& L, int e) {
  return reinterpret_cast<const PackedHeader*>(reinterpret_cast<const uint8_t*>(L.packed) +
                                               e * L.expert_bytes);
}

// One row block (16 rows x 64 k; this lane: rows g and g + 8, 16 k each) of a packed tile to
// 16-bit pairs in k order: og of row g, o8 of row g + 8.
template <int FMT, bool WIDE>
__device__ __forceinline__ void dequant_block(const int4& cw, uint32_t sc, uint32_t (&og)[8],
                                              uint32_t (&o8)[8]) {
  const uint32_t words[4] = {(uint32_t)cw.x, (uint32_t)cw.y, (uint32_t)cw.z, (uint32_t)cw.w};
  if constexpr (WIDE) {
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
    const uint32_t s2 = FMT == FMT_NV ? e4m3x2_to_f16x2(sc & 0xFFFFu) : mxenc2_to_f16x2(sc & 0xFFFFu);
    const uint32_t sg = bcast_lo(s2), s8 = bcast_hi(s2);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      uint32_t r0, r1, r2, r3;
      e2m1x8_to_f16x8(words[q], r0, r1, r2, r3);
      og[2 * q] = hmul2_u32(r0, sg);
      o8[2 * q] = hmul2_u32(r1, s8);
      og[2 * q + 1] = hmul2_u32(r2, sg);
      o8[2 * q + 1] = hmul2_u32(r3, s8);
    }
  }
}

__device__ __forceinline__ uint32_t ld_shared_u32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(addr));
  return v;
}

template <int FMT, bool SILU, int R, bool LOAD, int TOK>
__global__ void __launch_bounds__(kThreads, 1)
    k_ragged(const __grid_constant__ CUtensorMap tm, const RaggedParams p) {
  using S = Map<FMT, R, LOAD, TOK>;
  using TM = Tmem<R, TOK>;
  constexpr int TB = tile_bytes(FMT), NS = kNS, NW = S::NW, kSets = S::Sets;
  constexpr int kTok = TOK, kBBytes = S::BBytes, kBox = S::Box;
  constexpr uint32_t kTmemCols = TM::Cols, kBufs = TM::Bufs;
  const RaggedLaunch& L = p.L;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_u = smem_u32(smem_raw);
  const uint32_t base_u = (raw_u + 1023u) & ~1023u;
  uint8_t* base = smem_raw + (base_u - raw_u);
  const uint32_t sB = base_u, sW = base_u + S::OffW;
  const uint32_t full = base_u + S::OffBar, empty = full + 8 * NS;  // dequantised weights + tokens
  const uint32_t w_full = empty + 8 * NS, w_empty = w_full + 8 * NW;
  const uint32_t acc_full = w_empty + 8 * NW, acc_empty = acc_full + 16, drain = acc_empty + 16;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(base + S::OffBar + S::NumBars * 8);
  volatile int* abort = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* issued = abort + 1;  // packed stages requested, once the producer is done
  int2* s_tok = reinterpret_cast<int2*>(base + S::OffTok);
  Tiles T;
  T.E = L.E;
  T.start = reinterpret_cast<int*>(base + S::OffTab);
  T.first = T.start + L.E + 1;
  T.rows = reinterpret_cast<uint16_t*>(T.first + L.E + 1);
  T.of = T.rows + L.E + 1;

  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(full + 8 * s, 4 + (LOAD ? 128 : 1));  // a dequantiser set, the token copies
      mbar_init(empty + 8 * s, R);                    // the MMA threads
    }
    for (int s = 0; s < NW; ++s) {
      mbar_init(w_full + 8 * s, 1);
      mbar_init(w_empty + 8 * s, 4);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(acc_full + 8 * s, R);
      mbar_init(acc_empty + 8 * s, 8);
    }
    mbar_init(drain, 1);
    mbar_init(drain + 8, 1);
    *abort = *issued = 0;
  }
  if (warp == 2) tmem_alloc(smem_u32(tmem_slot), kTmemCols);
  fence_mbar_init();
  // The pre-pass lets this grid start only after its own wait for the kernels before it, so the
  // groups may be read (and the weights requested) at once; what the pre-pass writes is waited
  // for by the roles that read it.
  pdl_launch_dependents();
  bool bad = false;  // offsets out of order or out of range
  for (int e = threadIdx.x; e <= L.E; e += kThreads) {
    const int64_t v = __ldcg(L.offsets + e), c = v < 0 ? 0 : (v > L.pairs ? L.pairs : v);
    bad |= v != c;
    T.first[e] = (int)c;
  }
  __syncthreads();
  if (warp == 0) {  // token tiles of each group, summed up
    const int per = (L.E + 31) / 32, e0 = lane * per, e1 = min(e0 + per, L.E);
    int sum = 0;
    bool down = false;
    for (int e = e0; e < e1; ++e) {
      const int n = T.first[e + 1] - T.first[e];
      down |= n < 0;
      sum += (n + kTok - 1) / kTok;
    }
    down = __any_sync(0xffffffffu, down);  // then no tile at all: their number is bounded by order
    if (down) sum = 0;
    bad |= down;
    int run = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, run, o);
      if (lane >= o) run += u;
    }
    if (lane == 31) T.start[L.E] = run;
    run -= sum;
    for (int e = e0; e < e1; ++e) {
      T.start[e] = run;
      const int n = T.first[e + 1] - T.first[e];
      const int nt = down ? 0 : (n + kTok - 1) / kTok;
      // nearly equal tiles of whole MMA column blocks (at most kTok rows, so none is left empty)
      T.rows[e] = (uint16_t)(nt == 0 ? kTok : ((n + nt - 1) / nt + 15) & ~15);
      for (int t = run; t < run + nt && t < kTileTable; ++t) T.of[t] = (uint16_t)e;
      run += nt;
    }
  }
  if (blockIdx.x == 0 && bad) atomicExch(L.status, 6);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int tiles = T.start[L.E], KT = (int)L.KT, RT = (int)L.RT;
  const int64_t RGs = (RT + R - 1) / R;

  if (warp == 0) {
    // ---------------------------------------------------------- weight producer
    if (elect_one()) {
      const uint64_t pol = l2_evict_normal_policy();
      uint32_t iw = 0, pw = 0;
      int n = 0, hold = p.hold;
      bool ok = true;
      for (Walk w(RGs); ok && w.tile < tiles; w.next()) {
        const Item q = item_of(T, w.tile);
        const int rt0 = w.rg * R, nrt = R == 1 ? 1 : min(R, RT - rt0);
        const uint8_t* src = reinterpret_cast<const uint8_t*>(L.packed) + q.e * L.expert_bytes +
                             kHeaderBytes + (int64_t)rt0 * KT * TB;
        int kt = 0;
        do {
          // (the test hook outside the loop: a compare per step cost 2 of 43 us at 77 tokens)
          for (const int end = min(KT, kt + hold); kt < end; ++kt, src += TB) {
            if (!(ok = stage_wait(w_empty + 8 * iw, pw ^ 1u, abort, p))) break;
            mbar_expect_tx(w_full + 8 * iw, nrt * TB);
            for (int r = 0; r < nrt; ++r)
              bulk_g2s(sW + (iw * R + r) * TB, src + (int64_t)r * KT * TB, TB, w_full + 8 * iw, pol);
            if (++iw == NW) { iw = 0; pw ^= 1u; }
          }
          if (ok && kt < KT) {
            ok = L.withhold < 0;
            hold = kNoHold;
            const uint64_t t0 = globaltimer_ns();
            while (ok && globaltimer_ns() - t0 < kPauseNs) {}
          }
        } while (ok && kt < KT);
        n += kt;
        if (L.withhold) hold -= kt;
      }
      *issued = n;
    }
  } else if (warp == 1) {
    // ----------------------------------------------------------- token producer
    if (!LOAD && elect_one()) {
      const uint64_t pol = l2_evict_last_policy();
      uint32_t is = 0, ps = 0;
      bool ok = true;
      pdl_wait();
      for (Walk w(RGs); ok && w.tile < tiles; w.next()) {
        const Item q = item_of(T, w.tile);
        const int boxes = (q.n + kBox - 1) / kBox;
        for (int kt = 0; kt < KT; ++kt) {
          if (!(ok = stage_wait(empty + 8 * is, ps ^ 1u, abort, p))) break;
          const uint32_t dst = sB + is * kBBytes, bar = full + 8 * is;
          mbar_expect_tx(bar, (uint32_t)(boxes * kBox * 128));
          for (int b = 0; b < boxes; ++b)
            tma_load_2d(dst + b * kBox * 128, &tm, kt * kTileK, (int)q.i0 + b * kBox, bar, pol);
          if (++is == NS) { is = 0; ps ^= 1u; }
        }
      }
    }
  } else if (warp < kDeqWarp0) {
    // -------------------------------------------------------------- MMA issuers
    const int r = warp - 2;  // row tile
    if (r < R && elect_one()) {
      const uint32_t a0 = tmem + TM::A + r * 32, d0 = tmem + r * kTok;
      const uint64_t b0 = desc_sw128(sB);
      uint32_t is = 0, ps = 0, ic = 0, pc = 0;
      bool ok = true, ready = false;  // ready: the next stage was seen full
      for (Walk w(RGs); ok && w.tile < tiles; w.next()) {
        const Item q = item_of(T, w.tile);
        const bool live = SILU || r == 0 || w.rg * 2 + 1 < RT;  // not past an odd last row tile
        const bool wide = FMT == FMT_MX && header_of(L, q.e)->wide;
        const uint32_t idesc = (wide ? kIdescBF16 : kIdescF16) | ((uint32_t)((q.n + 15) >> 4) << 18);
        const uint32_t d = d0 + ic * R * kTok;  // ic: accumulator buffer
        if (!(ok = stage_wait(acc_empty + 8 * ic, pc ^ 1u, abort, p))) break;
        tc_fence_after();
        uint32_t acc = 0;
        for (int kt = 0; kt < KT; ++kt) {
          if (!ready && !(ok = stage_wait(full + 8 * is, ps, abort, p))) break;
          if (LOAD) fence_proxy_async_smem();  // the loaders' copies -> visible to the tensor core
          tc_fence_after();
          const uint32_t at = a0 + is * (R * 32), cur = empty + 8 * is;
          const uint64_t bd = b0 + is * (kBBytes >> 4);
          if (++is == NS) { is = 0; ps ^= 1u; }
          ready = mbar_test_wait(full + 8 * is, ps);  // answered while the MMAs are issued
          if (live) {
#pragma unroll
            for (int kk = 0; kk < kTileK / 16; ++kk) {  // 8 columns, 32 bytes per 16-element k step
              mma_f16_ts(d, at + 8 * kk, bd + 2 * kk, idesc, acc);
              acc = 1;
            }
          }
          mma_commit(cur);
        }
        if (!ok) break;
        mma_commit(acc_full + 8 * ic);
        if (++ic == kBufs) { ic = 0; pc ^= 1u; }
      }
      mma_commit(drain + 8 * r);  // every MMA issued has completed once this commit arrives
      const uint64_t t0 = globaltimer_ns();
      while (!mbar_try_wait(drain + 8 * r, 0) && globaltimer_ns() - t0 < kWaitNs) {}
    }
  } else if (warp < kDeqWarp0 + 4 * kSets) {
    // ------------------------------------------------------------- dequantisers
    // Set `set` takes the CTA's k steps set, set + kSets, ...; the warp of TMEM quarter jp two row
    // blocks (32 rows) for each accumulator, whose four scale bytes per lane are one word: blocks
    // 2jp and 2jp + 1 of row tile r, or (SiLU, R = 2) of tile jp / 2 its gate (r = 0) or up rows.
    const int set = (warp - kDeqWarp0) >> 2, jp = warp & 3, g = lane >> 2, t = lane & 3;
    const uint32_t ta = tmem + TM::A + ((uint32_t)(32 * jp) << 16);
    uint32_t iw = set, pw = 0, is = set, ps = 0;
    int kt = set;
    bool ok = true, wide = false, fresh = true;
    Walk w(RGs);
    while (w.tile < tiles && kt >= KT) { kt -= KT; w.next(); }
    while (w.tile < tiles) {
      if (FMT == FMT_MX && fresh) wide = header_of(L, item_of(T, w.tile).e)->wide != 0;
      const int nrt = R == 1 ? 1 : min(R, RT - w.rg * R);
      if (!(ok = warp_wait(w_full + 8 * iw, pw, abort, p))) break;
#pragma unroll
      for (int r = 0; r < R; ++r) {
        constexpr bool kSplit = SILU && R == 2;
        const int rt = kSplit ? jp >> 1 : r, j0 = kSplit ? r * 4 + (jp & 1) * 2 : 2 * jp;
        // (warp-uniform) past an odd last row tile there is nothing to read
        const bool live = rt < nrt;
        const uint32_t tb = sW + (iw * R + (live ? rt : 0)) * TB;
        const int4 cw0 = ld_shared_v4(tb + j0 * 512 + lane * 16);
        const int4 cw1 = ld_shared_v4(tb + (j0 + 1) * 512 + lane * 16);
        const uint32_t sc = ld_shared_u32(tb + scale_offset(FMT, j0, g, t));
        uint32_t og[2][8], o8[2][8];  // rows g and g + 8 of both row blocks
        if (FMT == FMT_MX && wide) {
          dequant_block<FMT, true>(cw0, sc, og[0], o8[0]);
          dequant_block<FMT, true>(cw1, sc >> 16, og[1], o8[1]);
        } else {
          dequant_block<FMT, false>(cw0, sc, og[0], o8[0]);
          dequant_block<FMT, false>(cw1, sc >> 16, og[1], o8[1]);
        }
        if (r == 0) {
          if (!(ok = warp_wait(empty + 8 * is, ps ^ 1u, abort, p))) break;
          tc_fence_after();
        }
        const uint32_t at = ta + (is * R + r) * 32;
        tmem_st_frag(at, og[0], o8[0]);
        tmem_st_frag(at + (16u << 16), og[1], o8[1]);
      }
      if (!ok) break;
      // The stores have taken every value computed from the packed stage, so its loads are done:
      // only now may the next copy overwrite it (an arrive placed after the conversions in the
      // source can be executed before them, while loads are under way).
      __syncwarp();
      if (lane == 0) mbar_arrive(w_empty + 8 * iw);
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(full + 8 * is);
      if ((iw += kSets) >= NW) { iw -= NW; pw ^= 1u; }
      if ((is += kSets) >= NS) { is -= NS; ps ^= 1u; }
      kt += kSets;
      fresh = kt >= KT;
      while (w.tile < tiles && kt >= KT) { kt -= KT; w.next(); }
    }
  } else if (warp < kEpiWarp0) {
    if constexpr (LOAD) {
      // ------------------------------------------------- loaders of gathered rows
      // Thread: 16-byte chunk c of rows r0, r0 + 16, ...; a row past the tile's tokens reads the
      // last one again (its products are not stored).  A wide expert's rows come from the
      // caller's bf16 activations.
      const int tid = (warp - (kDeqWarp0 + 4 * kSets)) * 32 + lane, c = tid & 7, r0 = tid >> 3;
      const uint32_t doff = (uint32_t)(r0 * 128 + ((c ^ (r0 & 7)) << 4));
      // where the two halves of a caller's chunk go (already in place in the pre-pass's rows)
      uint32_t hoff[2];
      for (int j = 0; j < 2; ++j) {
        const uint32_t o = pair_byte(c, j);
        hoff[j] = (uint32_t)(r0 * 128) + ((((o >> 4) ^ (uint32_t)(r0 & 7)) << 4) | (o & 15u));
      }
      uint32_t is = 0, ps = 0;
      bool ok = true;
      pdl_wait();
      for (Walk w(RGs); ok && w.tile < tiles; w.next()) {
        const Item q = item_of(T, w.tile);
        const bool wide = FMT == FMT_MX && header_of(L, q.e)->wide;
        const uint8_t* A = reinterpret_cast<const uint8_t*>(wide ? L.A : p.Ap);
        const int64_t ld = (wide ? L.lda : p.ldp) * 2;
        int row[kTok / 16];
#pragma unroll
        for (int i = 0; i < kTok / 16; ++i) {
          const int j = i * 16 + r0;
          row[i] = __ldcg(L.order + q.i0 + (j < q.n ? j : q.n - 1));
        }
#pragma unroll
        for (int i = 0; i < kTok / 16; ++i) {
          const bool in = row[i] >= 0 && row[i] < L.pairs;
          if (!in) atomicExch(L.status, 6);
          row[i] = in ? (int)((uint32_t)row[i] / (uint32_t)L.topk) : 0;
        }
        for (int kt = 0; kt < KT; ++kt) {
          if (!(ok = stage_wait(empty + 8 * is, ps ^ 1u, abort, p))) break;
          const uint32_t dst = sB + is * kBBytes;
          const int64_t k = (int64_t)kt * kTileK + c * 8;
          if (FMT == FMT_MX && wide) {
            const uint32_t bytes = k < L.K ? 8u : 0u;  // K is a multiple of 32
            const uint8_t* src = A + (k < L.K ? k * 2 : 0);
#pragma unroll
            for (int i = 0; i < kTok / 16; ++i)
              if (i * 16 < q.n) {
                cp_async8(dst + i * 2048 + hoff[0], src + row[i] * ld, bytes);
                cp_async8(dst + i * 2048 + hoff[1], src + row[i] * ld + 8, bytes);
              }
          } else {
#pragma unroll
            for (int i = 0; i < kTok / 16; ++i)
              if (i * 16 < q.n) cp_async16(dst + i * 2048 + doff, A + k * 2 + row[i] * ld);
          }
          cp_async_arrive(full + 8 * is);
          if (++is == NS) { is = 0; ps ^= 1u; }
        }
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
    }
  } else {
    // ----------------------------------------------------------------- epilogue
    // Warp qd of each group on TMEM lanes (weight rows) [32qd, 32qd + 32), 16 tokens at a time:
    // fragments from TMEM, scaled, rounded to bf16 and transposed through shared memory, from
    // where rows of contiguous columns are stored.
    const int eg = (warp - kEpiWarp0) >> 2, qd = warp & 3, t = lane & 3;
    constexpr int kTeam = R == 2 ? 256 : 128;  // threads that share a token table and a buffer
    const int tid = (R == 2 ? eg * 128 : 0) + qd * 32 + lane;
    __nv_bfloat16* C = reinterpret_cast<__nv_bfloat16*>(L.C);
    const bool vec = (uintptr_t)L.C % 16 == 0 && L.ldc % 8 == 0;
    const int64_t ncols = SILU ? L.seg_split : L.N;
    const int team = R == 2 ? 1 : 1 + eg;  // its named barrier
    auto team_sync = [&]() { asm volatile("bar.sync %0, %1;" ::"r"(team), "n"(kTeam) : "memory"); };
    // 16-byte piece of token j: 8 columns from column n on of its output row
    auto store_piece = [&](const int2* tok, int j, int64_t n, uint32_t from) {
      const int row = tok[j].x;
      if (row < 0 || n >= ncols) return;
      const int4 d = ld_shared_v4(from);
      __nv_bfloat16* dst = C + (int64_t)row * L.ldc + n;
      if (vec && n + 8 <= ncols) {
        *reinterpret_cast<int4*>(dst) = d;
      } else {
        const uint32_t w4[4] = {(uint32_t)d.x, (uint32_t)d.y, (uint32_t)d.z, (uint32_t)d.w};
#pragma unroll
        for (int b = 0; b < 8; ++b)
          if (n + b < ncols)
            reinterpret_cast<uint16_t*>(dst)[b] = (uint16_t)(w4[b >> 1] >> ((b & 1) * 16));
      }
    };
    // scales of this lane's tokens 2t, 2t + 1 of a chunk and the same 8 on
    auto scales = [&](const int2* tok, float (&rs)[4]) {
      const int4 a = *reinterpret_cast<const int4*>(tok + 2 * t);
      const int4 b = *reinterpret_cast<const int4*>(tok + 8 + 2 * t);
      rs[0] = __int_as_float(a.y);
      rs[1] = __int_as_float(a.w);
      rs[2] = __int_as_float(b.y);
      rs[3] = __int_as_float(b.w);
    };
    uint32_t ic = 0, pc = 0, chunk = 0, odd = 0;
    bool ok = true;
    pdl_wait();
    // this thread's token of the item: its pair, fetched an item ahead
    Walk w(RGs);
    int pair = 0;
    auto fetch = [&]() {
      if ((L.scatter || LOAD) && w.tile < tiles) {
        const Item q = item_of(T, w.tile);
        pair = tid < q.n ? __ldcg(L.order + q.i0 + tid) : 0;
      }
    };
    fetch();
    while (ok && w.tile < tiles) {
      const Item q = item_of(T, w.tile);
      const int rt0 = w.rg * R, nrt = R == 1 ? 1 : min(R, RT - rt0);
      const PackedHeader* hdr = header_of(L, q.e);
      const float f0 = hdr->factor[0], f1 = hdr->factor[1];
      const bool wide = FMT == FMT_MX && hdr->wide;
      int2* tok = s_tok + ((R == 2 ? 0 : eg * 2) + odd) * kTok;
      odd ^= 1u;
      if (tid < kTok) {
        int row = -1;
        float rs = 1.0f;
        if (tid < q.n) {
          row = (int)q.i0 + tid;
          bool in = true;
          if (L.scatter || LOAD) in = pair >= 0 && pair < L.pairs;
          if (!in) atomicExch(L.status, 6);
          if (!wide && in) rs = __ldcg(p.rowscale + (LOAD ? (int64_t)((uint32_t)pair / (uint32_t)L.topk) : row));
          if (L.scatter) row = in ? pair : -1;
        }
        tok[tid] = make_int2(row, __float_as_int(rs));
      }
      w.next();
      fetch();
      // behind it the table is written, and the buffer of the item before read
      if (!(ok = team_wait<kTeam>(team, acc_full + 8 * ic, pc, abort, p))) break;
      tc_fence_after();
      const uint32_t ta = tmem + ic * R * kTok + ((uint32_t)(qd * 32) << 16);
      if constexpr (R == 2) {
        // Group eg: row tile eg (SiLU: every other chunk, both accumulators of it).
        constexpr int kCols = SILU ? 128 : 256, kRowB = kCols * 2 + 16;
        const uint32_t sX = base_u + S::OffX;
        if (SILU || eg < nrt) {
          const int64_t split = SILU ? 0 : L.seg_split - (int64_t)(rt0 + eg) * 128 - qd * 32;
          for (int c = SILU ? eg : 0; c * 16 < q.n; c += SILU ? 2 : 1) {
            uint32_t v[2][8], u[2][8];  // weight rows [0, 16), [16, 32) of the warp's; SiLU: u of up
            const uint32_t tc = ta + c * 16 + (SILU ? 0 : eg * kTok);
            tmem_ld_frag(tc, v[0]);
            tmem_ld_frag(tc + (16u << 16), v[1]);
            if constexpr (SILU) {
              tmem_ld_frag(tc + kTok, u[0]);
              tmem_ld_frag(tc + kTok + (16u << 16), u[1]);
            }
            float rs[4];
            scales(tok + c * 16, rs);
            tmem_wait_frags(v[0], v[1]);
            if constexpr (SILU) tmem_wait_frags(u[0], u[1]);
            uint32_t o[2][4];
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                float y[2];
#pragma unroll
                for (int z = 0; z < 2; ++z) {
                  const float s = rs[z + (i >> 1) * 2];
                  if constexpr (SILU) {
                    y[z] = silu_f(__uint_as_float(v[h][2 * i + z]) * s * f0) *
                           (__uint_as_float(u[h][2 * i + z]) * s * f1);
                  } else {
                    const float f = h * 16 + (lane >> 2) + (i & 1) * 8 < split ? f0 : f1;
                    y[z] = __uint_as_float(v[h][2 * i + z]) * s * f;
                  }
                }
                o[h][i] = pack_bf16(y[0], y[1]);
              }
#pragma unroll
            for (int th = 0; th < 2; ++th)
              stmatrix_t4(sX + (c * 16 + th * 8 + (lane & 7)) * kRowB +
                              ((SILU ? 0 : eg * 128) + qd * 32 + (lane >> 3) * 8) * 2,
                          o[0][2 * th], o[0][2 * th + 1], o[1][2 * th], o[1][2 * th + 1]);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(acc_empty + 8 * ic);  // the MMAs of the next item may begin
        team_sync();
        constexpr int kPieces = kCols / 8;
#pragma unroll 4
        for (int i = tid; i < q.n * kPieces; i += kTeam) {
          const int j = i / kPieces, c8 = i % kPieces;
          store_piece(tok, j, (int64_t)rt0 * (kCols / 2) + c8 * 8, sX + j * kRowB + c8 * 16);
        }
      } else {
        // Group eg: every other chunk of the item's tokens.
        constexpr int kCols = SILU ? 64 : 128, kRowB = kCols * 2 + 16, kPieces = kCols / 8;
        const uint32_t sX = base_u + S::OffX + eg * S::XGroup, sT = sX + (SILU ? 8192 : 0);
        const bool up = SILU && qd >= 2;
        const int64_t n0 = (int64_t)rt0 * kCols, split = L.seg_split - n0 - qd * 32;
        for (int c = eg; c * 16 < q.n; c += 2, ++chunk) {
          const uint32_t buf = sT + (chunk & 1) * (16 * kRowB);
          uint32_t v[2][8];
          tmem_ld_frag(ta + c * 16, v[0]);
          tmem_ld_frag(ta + c * 16 + (16u << 16), v[1]);
          float rs[4], x[2][8];
          scales(tok + c * 16, rs);
          tmem_wait_frags(v[0], v[1]);
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const bool second = SILU ? up : h * 16 + (lane >> 2) + ((i >> 1) & 1) * 8 >= split;
              x[h][i] = __uint_as_float(v[h][i]) * rs[(i & 1) + (i >> 2) * 2] * (second ? f1 : f0);
            }
          if constexpr (SILU) {
            // warps 0-1 hold gate rows, warps 2-3 the matching up rows in the same places: of
            // every 16 tokens the gate warps finish the first 8 and the up warps the others
            const uint32_t ex = sX + (chunk & 1) * 4096 + lane * 16;
#pragma unroll
            for (int h = 0; h < 2; ++h)
              st_shared_v4(ex + (qd * 2 + h) * 512, __float_as_uint(up ? x[h][0] : x[h][4]),
                           __float_as_uint(up ? x[h][1] : x[h][5]),
                           __float_as_uint(up ? x[h][2] : x[h][6]),
                           __float_as_uint(up ? x[h][3] : x[h][7]));
            team_sync();
            uint32_t o[4];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int4 z = ld_shared_v4(ex + ((qd ^ 2) * 2 + h) * 512);
              const float zz[4] = {__int_as_float(z.x), __int_as_float(z.y), __int_as_float(z.z),
                                   __int_as_float(z.w)};
              float a[4];
#pragma unroll
              for (int i = 0; i < 4; ++i)
                a[i] = up ? silu_f(zz[i]) * x[h][4 + i] : silu_f(x[h][i]) * zz[i];
              o[2 * h] = pack_bf16(a[0], a[1]);
              o[2 * h + 1] = pack_bf16(a[2], a[3]);
            }
            stmatrix_t4(buf + ((up ? 8 : 0) + (lane & 7)) * kRowB + ((qd & 1) * 32 + (lane >> 3) * 8) * 2,
                        o[0], o[1], o[2], o[3]);
          } else {
#pragma unroll
            for (int th = 0; th < 2; ++th)
              stmatrix_t4(buf + (th * 8 + (lane & 7)) * kRowB + (qd * 32 + (lane >> 3) * 8) * 2,
                          pack_bf16(x[0][4 * th], x[0][4 * th + 1]),
                          pack_bf16(x[0][4 * th + 2], x[0][4 * th + 3]),
                          pack_bf16(x[1][4 * th], x[1][4 * th + 1]),
                          pack_bf16(x[1][4 * th + 2], x[1][4 * th + 3]));
          }
          team_sync();
#pragma unroll
          for (int i = 0; i < 16 * kPieces / 128; ++i) {
            const int j = (i * 128 + tid) / kPieces, c8 = (i * 128 + tid) % kPieces;
            store_piece(tok + c * 16, j, n0 + c8 * 8, buf + j * kRowB + c8 * 16);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(acc_empty + 8 * ic);
      }
      if (++ic == kBufs) { ic = 0; pc ^= 1u; }
    }
  }

  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
  if (threadIdx.x == 0 && *abort) {
    // Some role gave up, perhaps not the producers: shared memory is kept until the copies under way
    // have landed.  The packed stages have a barrier of their own each; the token stages' barriers
    // also count the dequantisers, who may have left, so the last of those copies get a
    // millisecond, a thousand times what one takes.
    atomicExch(L.status, 5);
    const int n = *issued;
    for (int k = n > NW ? n - NW : 0; k < n; ++k)
      mbar_wait_bounded(w_full + 8 * (k % NW), (uint32_t)(k / NW) & 1u, kWaitNs);
    const uint64_t t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < 1000000ull) {}
  }
}

// Activation pre-pass: A'[i][k] = A[row(i)][k] * 2^-p in f16, p the power of two of the row's
// largest magnitude (act_pow2), rowscale[i] = 2^p, the k of each 64 in the MMA's order.  One warp
// per row: grouped row i (a row of a `wide` expert is copied as bf16 with scale 1), or, per_token,
// the caller's row i.  Bound by memory: a row of up to HELD x 32 granules of 8 values stays in
// registers between its maximum and its conversion (a block of 128 threads per row took 38 us for
// 32768 rows of 768).
constexpr int kPrepThreads = 256;
template <int HELD>
__global__ void __launch_bounds__(kPrepThreads) k_ragged_prep(const RaggedLaunch L, int64_t rows,
                                                              int64_t ldp, int per_token,
                                                              __half* __restrict__ Ap,
                                                              float* __restrict__ rowscale) {
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t i = (int64_t)blockIdx.x * (kPrepThreads / 32) + (threadIdx.x >> 5);
  if (i >= rows) return;
  const int64_t grouped = per_token ? rows : (int64_t)__ldcg(L.offsets + L.E);
  int64_t m = i;
  if (L.gather && !per_token) {
    const int pr = __ldcg(L.order + i);
    const bool in = pr >= 0 && pr < L.pairs;
    if (!in && lane == 0) atomicExch(L.status, 6);
    m = in ? pr / L.topk : 0;
  }
  const uint4* row = reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(L.A) + m * L.lda);
  // granule k in the MMA's order, as two halves; granules past K are zeros
  uint8_t* dst = reinterpret_cast<uint8_t*>(Ap + i * ldp);
  auto put = [&](int k, const uint4& v) {
    uint8_t* tile = dst + (int64_t)(k >> 3) * 128;
    *reinterpret_cast<uint2*>(tile + pair_byte(k & 7, 0)) = make_uint2(v.x, v.y);
    *reinterpret_cast<uint2*>(tile + pair_byte(k & 7, 1)) = make_uint2(v.z, v.w);
  };
  const int ng = (int)(L.K / 8), ngp = (int)(ldp / 8);
  const uint4 zero = make_uint4(0, 0, 0, 0);
  uint4 held[HELD];
#pragma unroll
  for (int h = 0; h < HELD; ++h) held[h] = h * 32 + lane < ng ? row[h * 32 + lane] : zero;
  if (i >= grouped) return;  // a pair in no group
  if (L.fmt == FMT_MX && !per_token) {
    int e = 0;
    for (int b = lane; b < L.E; b += 32)
      if (__ldcg(L.offsets + b) <= i && i < __ldcg(L.offsets + b + 1)) e = b;
    e = __reduce_max_sync(0xffffffffu, e);
    if (header_of(L, e)->wide) {
      for (int k = lane; k < ngp; k += 32) put(k, k < ng ? row[k] : zero);
      if (lane == 0) rowscale[i] = 1.0f;
      return;
    }
  }
  int mx = 0;
  auto grow = [&](const uint4& v) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    mx = max(mx, act_maxmag8(w));
  };
#pragma unroll
  for (int h = 0; h < HELD; ++h) grow(held[h]);
#pragma unroll 4
  for (int k = HELD * 32 + lane; k < ng; k += 32) grow(row[k]);
  mx = __reduce_max_sync(0xffffffffu, mx);
  const int p = act_pow2(mx);
  auto convert = [&](int k, const uint4& v) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    put(k, act_granule_f16(w, p));
  };
#pragma unroll
  for (int h = 0; h < HELD; ++h)
    if (h * 32 + lane < ngp) convert(h * 32 + lane, held[h]);
#pragma unroll 4
  for (int k = HELD * 32 + lane; k < ngp; k += 32) convert(k, k < ng ? row[k] : zero);
  if (lane == 0) rowscale[i] = pow2f(p);
}

// Weighted sum of each token's pairs, in slot order, in fp32; 8 columns per thread, a block per
// token and 2048 columns.  The loads of 8 slots are in flight together, those of pairs in no group
// too (what their rows hold is not used): one after another, behind the test of each slot's id,
// 4096 tokens x top-8 x 2048 columns took 39 us, 25 now (5.5 TB/s).  Bound by memory.  D is bf16: each
// pair's output is rounded once as a product of its own would be (in fp32 its 134 MB written and
// read there would be twice that), and the sum is rounded once more.
constexpr int kCombineThreads = 256;
__global__ void __launch_bounds__(kCombineThreads) k_combine(
    const __nv_bfloat16* __restrict__ D, int topk, int N, int64_t ldd,
    const int32_t* __restrict__ ids, int E, const float* __restrict__ weights,
    __nv_bfloat16* __restrict__ out, int64_t ldo, int vec) {
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t m = blockIdx.x;
  const int n0 = (int)(blockIdx.y * blockDim.x + threadIdx.x) * 8;
  const bool live = n0 < N;
  float acc[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  // D's rows are padded to 8 columns (what lies in the padding is not stored)
  const __nv_bfloat16* src = D + m * topk * ldd + (live ? n0 : 0);
  ids += m * topk;
  weights += m * topk;
  for (int j0 = 0; j0 < topk; j0 += 8) {
    // lane j: slot j0 + j
    const bool slot = lane < 8 && j0 + lane < topk;
    const int id = slot ? __ldg(ids + j0 + lane) : -1;
    const float wl = slot ? __ldg(weights + j0 + lane) : 0.0f;
    uint4 v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j)
      v[j] = j0 + j < topk ? __ldcs(reinterpret_cast<const uint4*>(src + (j0 + j) * ldd)) : make_uint4(0, 0, 0, 0);
    const uint32_t in = __ballot_sync(0xffffffffu, id >= 0 && id < E);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float w = __shfl_sync(0xffffffffu, wl, j);
      if (in >> j & 1) {
        const uint32_t x[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          acc[2 * c] += w * __uint_as_float(x[c] << 16);
          acc[2 * c + 1] += w * __uint_as_float(x[c] & 0xFFFF0000u);
        }
      }
    }
  }
  if (!live) return;
  __nv_bfloat16* dst = out + m * ldo + n0;
  if (vec && n0 + 8 <= N) {
    *reinterpret_cast<uint4*>(dst) = make_uint4(pack_bf16(acc[0], acc[1]), pack_bf16(acc[2], acc[3]),
                                                pack_bf16(acc[4], acc[5]), pack_bf16(acc[6], acc[7]));
  } else {
    for (int c = 0; c < 8 && n0 + c < N; ++c) dst[c] = __float2bfloat16_rn(acc[c]);
  }
}

}  // namespace

namespace {

cudaLaunchConfig_t pdl_config(cudaLaunchAttribute* at, dim3 grid, int threads, int smem, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = s;
  at->id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at->val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cfg;
}

template <int FMT, bool SILU, int R, bool LOAD, int TOK>
cudaError_t launch_main(const CUtensorMap& tm, const RaggedParams& p, cudaStream_t s, RaggedShape* shape) {
  using S = Map<FMT, R, LOAD, TOK>;
  static int done[64] = {0};
  const cudaError_t e =
      set_up_kernel(k_ragged<FMT, SILU, R, LOAD, TOK>, (size_t)S::smem(kMaxGroups), done);
  if (e != cudaSuccess) return e;
  // at most one partial token tile per group in use
  const int64_t groups = p.L.pairs < p.L.E ? p.L.pairs : p.L.E;
  const int64_t most = (groups + p.L.pairs / TOK) * ((p.L.RT + R - 1) / R);
  const int grid = (int)(sm_count() < most ? sm_count() : most);
  *shape = {grid, kThreads / 32, TOK, most};
  cudaLaunchAttribute at;
  const cudaLaunchConfig_t cfg = pdl_config(&at, dim3((unsigned)grid), kThreads, S::smem(p.L.E), s);
  return cudaLaunchKernelEx(&cfg, k_ragged<FMT, SILU, R, LOAD, TOK>, tm, p);
}

template <int FMT, bool SILU>
cudaError_t launch_fmt(const CUtensorMap& tm, const RaggedParams& p, bool two, bool many, bool load,
                       cudaStream_t s, RaggedShape* shape) {
  if (!two) return launch_main<FMT, SILU, 1, false, 64>(tm, p, s, shape);
  if (!many) return launch_main<FMT, SILU, 2, false, 64>(tm, p, s, shape);
  return load ? launch_main<FMT, SILU, 2, true, 128>(tm, p, s, shape)
              : launch_main<FMT, SILU, 2, false, 128>(tm, p, s, shape);
}

}  // namespace

size_t ragged_act_bytes(int64_t pairs, int64_t KT) {
  return (size_t)((pairs * 4 + 255) / 256 * 256 + pairs * KT * kTileK * 2);
}

cudaError_t launch_ragged(const RaggedLaunch& L, cudaStream_t s, RaggedShape* shape) {
  auto enc = tensor_map_encoder();
  if (!enc) return cudaErrorNotSupported;
  RaggedParams p;
  p.L = L;
  p.ldp = L.KT * kTileK;
  float* rowscale = reinterpret_cast<float*>(L.act);
  __half* ap = reinterpret_cast<__half*>(reinterpret_cast<uint8_t*>(L.act) + (L.pairs * 4 + 255) / 256 * 256);
  p.rowscale = rowscale;
  p.Ap = ap;
  p.wait_ns = L.wait_ns ? L.wait_ns : kWaitNs;
  p.hold = L.withhold == 0 ? kNoHold : L.withhold > 0 ? L.withhold - 1 : -1 - L.withhold;
  // The rules below were measured on 128 experts, top-8, gate_up 1536 x 2048 NVFP4 ("A") and 24
  // experts, top-3, gate_up 2880 x 2592 MXFP4 ("B"), us:
  // One row tile per item while every item gets an SM of its own, so that an SM's share of the
  // weights is the least (1 token, A: 10.6, 12.2 with two; B: 12.5 and 14.1); else two, which share
  // the token tile (2 tokens, A: 13.0, 16.6 with one; 77: 44 and 62).
  const int64_t groups = L.pairs < L.E ? L.pairs : L.E;
  const bool two = groups * L.RT > sm_count();
  // Tiles of 128 rows from 64 rows per group on (64 rows, A: 70, 85 with tiles of 64; B: 38 and 43;
  // 32 rows, A: 62.6 and 63.8; 19 rows, B: 31.3 and 30.2).
  const bool many = two && L.pairs >= 64 * groups;
  // Gathered rows: the pre-pass writes them in group order while that is little data (3063 rows, B:
  // 52.2 either way; 4096 rows, A: 64), else it converts each token once and the loaders gather (6144
  // rows, B: 83.1, 84.6 in group order; 8192 rows, A: 69 and 78; 32768: 166 and 189).
  const bool load = L.gather && L.topk > 1 && many && L.pairs * L.K > (8 << 20);
  const int64_t rows = load ? L.pairs / L.topk : L.pairs;
  // the converted rows as a 2-D tensor: reads past the last row return zeros
  CUtensorMap tm;
  const cuuint64_t dims[2] = {(cuuint64_t)p.ldp, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)p.ldp * 2};
  const cuuint32_t box[2] = {(cuuint32_t)kTileK, (cuuint32_t)(many ? 32 : 16)};
  const cuuint32_t estr[2] = {1, 1};
  if (enc(&tm, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, ap, dims, strides, box, estr,
          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
          CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return cudaErrorInvalidValue;
  cudaLaunchAttribute at;
  constexpr int kRows = kPrepThreads / 32;
  const cudaLaunchConfig_t cfg =
      pdl_config(&at, dim3((unsigned)((rows + kRows - 1) / kRows)), kPrepThreads, 0, s);
  cudaError_t e = L.K <= 1024
                      ? cudaLaunchKernelEx(&cfg, k_ragged_prep<4>, L, rows, p.ldp, load ? 1 : 0, ap, rowscale)
                      : cudaLaunchKernelEx(&cfg, k_ragged_prep<8>, L, rows, p.ldp, load ? 1 : 0, ap, rowscale);
  if (e != cudaSuccess) return e;
  if (L.fmt == FMT_NV) return L.silu ? launch_fmt<FMT_NV, true>(tm, p, two, many, load, s, shape)
                                     : launch_fmt<FMT_NV, false>(tm, p, two, many, load, s, shape);
  return L.silu ? launch_fmt<FMT_MX, true>(tm, p, two, many, load, s, shape)
                : launch_fmt<FMT_MX, false>(tm, p, two, many, load, s, shape);
}

cudaError_t launch_combine(const void* D, int64_t M, int topk, int64_t N, int64_t ldd,
                           const int32_t* ids, int E, const float* weights, void* out,
                           int64_t ldo, cudaStream_t s) {
  const int64_t pieces = (N + 7) / 8;
  const int threads = (int)(pieces < kCombineThreads ? (pieces + 31) / 32 * 32 : kCombineThreads);
  const dim3 grid((unsigned)M, (unsigned)((pieces + threads - 1) / threads));
  const int vec = (uintptr_t)out % 16 == 0 && ldo % 8 == 0;
  cudaLaunchAttribute at;
  const cudaLaunchConfig_t cfg = pdl_config(&at, grid, threads, 0, s);
  return cudaLaunchKernelEx(&cfg, k_combine, reinterpret_cast<const __nv_bfloat16*>(D), topk, (int)N,
                            ldd, ids, E, weights, reinterpret_cast<__nv_bfloat16*>(out), ldo, vec);
}

}  // namespace vt
