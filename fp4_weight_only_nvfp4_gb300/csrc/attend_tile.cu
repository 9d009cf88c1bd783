// Causal attention of chunks of rows over the paged NVFP4 cache, on the 5th-generation tensor cores.
//
//   S = Q K^T,  P = 2^(S - m),  O = O + P V,  out = O / sum P
// A tile is the rows of one key/value head: tokens x its query heads, 128 rows an MMA; two such row
// tiles (one at head_dim 256) share each block of keys, so that a block is turned into f16 once for 256
// rows and one row tile's softmax runs beside the other's products.  Bound by the tensor cores for
// long chunks; for a few rows by the cache's bytes and their conversion.
//
// One persistent CTA per SM:
//   softmax warps  4 per row tile, a thread per row: Q to shared memory (f16, times a power of two per
//                  row), then per block the row's maximum, the probabilities (written over the
//                  scores in TMEM as the A operand of the second product) and their sum; at the end
//                  O to the output.  O is scaled only where a row's maximum rose by more than 2^8: until then the
//                  sums stay on the older one, which f16 has room for.
//   K, V warps     4 each: codes and scales straight from the pages to registers a block ahead,
//                  then f16 (c * s, exact) into shared memory, K as [token][d], V as [d][token]
//                  (both K-major, 128-byte swizzle).
//   MMA warp       one thread issues every product.
// The tiles' blocks of keys, times the heads, stand in one line that is shared out evenly over the
// CTAs; the parts of a tile that CTAs share are joined by the CTA that comes last.  Each (tile,
// head) stands there with kLead units more than its blocks, for its start and end.
//
// Measured: a prompt of 8192 rows, 32 heads on 4 of 128: 502 us, 1095 TFLOP/s of its causal half, the
// tensor pipe 48 % active; the products of one row tile wait for its softmax and
// share the shared memory with the conversion's stores.  Five chunks of up to 900 rows behind 2500 keys, 64 heads
// on 8 of 64, window 512 (five blocks a tile): 105 us, half of it a tile's start and end.  4096 rows, 24 heads on 4 of 256: 400 us.
//
// The roles' loops together are about as long as the instruction cache, so code in them counts even where it is not
// entered: with 30 instructions more in the V warps' 8192 rows took 565 us instead of 537, and where the K warps' grew 635, with
// 1.7 warps an issue waiting for instructions instead of 0.5.  So what a wait does when it is not over at once is a function
// of its own, and a pass that can be a loop is one (565 to 513 us; 0.4 warps).
//
// Every wait inside the CTA is bounded (2 s); one that gives up sets the status word and ends every role.
#include <cuda_bf16.h>

#include "actq.cuh"
#include "attend.cuh"
#include "common.cuh"
#include "handle.h"
#include "kernels.h"
#include "kv.cuh"
#include "tc.cuh"

namespace vt {

namespace {

constexpr uint64_t kWaitNs = 2000000000ull, kPauseNs = 1000000ull;
constexpr uint32_t kNoHold = 0xFFFFFFFFu;
// (8192 rows, 32 heads on 4: 634 us with 4, 602 with 6, 615 with 9)
constexpr int kLead = 6;

template <int D>
struct TileCfg {
  static constexpr int kRowTiles = D == 256 ? 1 : 2;
  static constexpr int kSBufs = D == 256 ? 2 : 1;         // score buffers of a row tile
  static constexpr int kKeys = D == 256 ? 64 : 128;       // keys of a block
  static constexpr int kSoftWarps = 4 * kRowTiles;
  // 16 warps for two row tiles: a 17th would leave every thread 96 registers, and the softmax takes all
  // of its 128 (a spill goes into an L1 that the shared memory leaves next to nothing).
  static constexpr int kVWarps = kRowTiles == 2 ? 3 : 4;
  static constexpr int kWarpK = kSoftWarps, kWarpV = kWarpK + 4, kWarpMma = kWarpV + kVWarps;
  static constexpr int kThreads = (kWarpMma + 1) * 32;
  static constexpr int kQBytes = 128 * D * 2;             // a row tile
  static constexpr int kKvBytes = kKeys * D * 2;          // a block of K or V
  static constexpr int kStages = 2;
  static constexpr int kOffK = kRowTiles * kQBytes;
  static constexpr int kOffV = kOffK + kStages * kKvBytes;
  static constexpr int kOffMeta = kOffV + kStages * kKvBytes;
  // Conversion goes in jobs of 64 values per lane: 16 tokens of 128 columns, or 32 of 64.
  static constexpr int kAllJobs = kKeys * D / 2048;       // of a block of K or V
  static constexpr int kKJobs = kAllJobs / 4, kVJobs = (kAllJobs + kVWarps - 1) / kVWarps;
  // TMEM columns: scores (P over them), then O
  static constexpr int kTmemO = 256;
  static constexpr int kRows = 128 * kRowTiles;
  static constexpr int kPartFloats = kRows * (D + 4);     // O in columns of 4, then m, l, any
};

constexpr int kNanAtBorder = 16;
struct TileShared {
  int64_t scan[32];
  int64_t seq_first[32 * 16 + 1];
  int64_t before;      // the units before this CTA's first tile
  int64_t G, total;    // CTAs in use, units in all
  int b, i;            // its tile
  int last;
  int2 v_seen[4][2];                // of each V warp, of two segments: its blocks that every row of the tile sees
  // of the segments under way, that of number n in place n & 7: n + 1 where the values hold a NaN scale (see nan_columns)
  int nan_seg[8], nan_what[8][17];
  float half_m[128], half_l[128];  // of the row tile's second half of blocks
  int half_any[128];
  uint32_t tmem;
  int abort;
  alignas(8) uint64_t bars[24];
  alignas(16) uint8_t walk[8 * 96];  // of each softmax warp
  alignas(16) int row[256][4];       // of each softmax thread: first key, end of the keys, factor of the scores, sink
  float value[8];                    // of each softmax warp: the values' global
};

struct TileParams {
  AttendLaunch a;
  int G;
  int tokens;     // of a row tile: 128 / group
  uint32_t by_group;  // floor(2^32 / group) + 1: quotients of small numbers by it
  float* parts;
  uint64_t wait_ns;
  uint32_t hold;      // test hook: the block before which the K warps stop,
  int pause;          // or pause
};

// A sequence as this kernel takes it: n = 0 where the row kernel does.
__device__ __forceinline__ AttendSeq tile_seq(const AttendLaunch& a, int64_t b) {
  AttendSeq q = load_seq(a, b);
  if (few_rows(a, q.n)) q.n = 0;
  return q;
}

// Blocks of keys of a sequence's i-th tile: [first, first + count).
template <int D>
__device__ __forceinline__ void tile_blocks(const AttendLaunch& a, const AttendSeq& q, int i, int per_tile, int* first, int* count) {
  constexpr int KB = TileCfg<D>::kKeys;
  const int r0 = i * per_tile, r1 = min(q.n, r0 + per_tile);
  const int64_t past = (int64_t)q.len - q.n;
  const int64_t hi = past + r1;                                // keys that its last row sees
  int64_t lo = a.window > 0 ? past + r0 - a.window + 1 : 0;    // the first key that its first row sees
  if (lo < 0) lo = 0;
  *first = (int)(lo / KB);
  *count = hi > 0 && hi > lo ? (int)((hi + KB - 1) / KB) - *first : 0;
}

// A run of blocks of one (tile, head), walked by every role on its own.
template <int D>
struct Walk {
  AttendSeq q;
  int b, i, h;
  int first, count;   // the tile's blocks
  int at, end;        // this segment: blocks [at, end) of them, counted from first
  int64_t seg0;       // unit of block 0
  int64_t left;       // units of the CTA from the (tile, head)'s first, or the CTA's own first, on
  int no;             // segments before this one
  static __device__ __forceinline__ int per_tile(const TileParams& p) { return p.tokens * TileCfg<D>::kRowTiles; }
  // The CTA's first segment; false if there is no block in its units.
  __device__ __forceinline__ bool start(const TileParams& p, const TileShared& sh, int64_t u0, int64_t u1) {
    b = sh.b;
    i = sh.i;
    q = tile_seq(p.a, b);
    tile_blocks<D>(p.a, q, i, per_tile(p), &first, &count);
    const int64_t r = u0 - sh.before;
    h = (int)(r / (count + kLead));
    const int off = (int)(r - (int64_t)h * (count + kLead));
    seg0 = u0 - off + kLead;
    left = u1 - u0 + off;
    no = 0;
    return cut(off);
  }
  __device__ __forceinline__ bool cut(int off) {
    at = max(off - kLead, 0);
    end = (int)min((int64_t)count, left - kLead);
    return end > at;
  }
  // To the CTA's next segment; false at its end.
  __device__ __forceinline__ bool next(const TileParams& p) {
    left -= count + kLead;
    if (left <= 0) return false;
    ++no;
    seg0 += count + kLead;
    if (++h == p.a.cache.heads) {
      h = 0;
      do {
        ++i;
        while ((int64_t)i * per_tile(p) >= q.n) {
          if (++b >= p.a.B) { left = 0; return false; }
          q = tile_seq(p.a, b);
          i = 0;
        }
        tile_blocks<D>(p.a, q, i, per_tile(p), &first, &count);
      } while (count == 0);
    }
    return cut(0);
  }
  __device__ __forceinline__ int row_tiles(const TileParams& p) const {
    return TileCfg<D>::kRowTiles == 2 && q.n - i * per_tile(p) > p.tokens ? 2 : 1;
  }
  // One row tile of the two: its blocks go to both in turn, and their halves are joined at the end.
  __device__ __forceinline__ bool halved(const TileParams& p) const {
    return TileCfg<D>::kRowTiles == 2 && row_tiles(p) == 1;
  }
  __device__ __forceinline__ bool whole() const { return at == 0 && end == count; }
};

__device__ __forceinline__ void mma_f16_ta(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                           uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
      "%12, %13, %14, %15};" ::"r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]),
      "r"(v[7]), "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&v)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%8], {%0, %1, %2, %3, %4, %5, %6, %7};" ::"r"(v[0]),
               "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(taddr)
               : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
      "%12, %13, %14, %15}, [%16];\n tcgen05.wait::ld.sync.aligned;"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
        "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&v)[32]) {
  uint32_t a[16], b[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) a[i] = v[i], b[i] = v[16 + i];
  tmem_st16(taddr, a);
  tmem_st16(taddr + 16, b);
}
// Bounded wait; the warp sleeps in the barrier for up to 20 us at a time, so that those that wait take
// no issue slots from those that work.  What follows the first sleep is called, not inlined, for the code's size.
__device__ __forceinline__ bool try_wait_long(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n"
      " selp.u32 %0, 1, 0, p;\n}"
      : "=r"(ok)
      : "r"(bar), "r"(parity), "r"(20000)
      : "memory");
  return ok != 0;
}
__device__ __noinline__ bool wait_slow(uint32_t bar, uint32_t parity, volatile int* abort, uint64_t limit_ns) {
  const uint64_t t0 = globaltimer_ns();
  while (true) {
    if (try_wait_long(bar, parity)) return true;
    if (*abort) return false;
    if (globaltimer_ns() - t0 > limit_ns) {
      *abort = 1;
      return false;
    }
  }
}
__device__ __forceinline__ bool wait_for(uint32_t bar, uint32_t parity, volatile int* abort, uint64_t limit_ns) {
  if (try_wait_long(bar, parity)) return true;
  return wait_slow(bar, parity, abort, limit_ns);
}
__device__ __noinline__ void pause() {
  const uint64_t t0 = globaltimer_ns();
  while (globaltimer_ns() - t0 < kPauseNs) __nanosleep(1000);
}
// One answer for the warp.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int* abort, uint64_t limit_ns) {
  return __all_sync(0xffffffffu, wait_for(bar, parity, abort, limit_ns));
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

constexpr uint32_t idesc_f16(int n) { return (1u << 4) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(128 >> 4) << 24); }

// Blocks of keys [lo, hi) that every row of the tile sees (none where lo >= hi).
template <int D>
__device__ __forceinline__ void seen_by_all(const TileParams& p, const Walk<D>& w, int* lo, int* hi) {
  constexpr int KB = TileCfg<D>::kKeys;
  const int r0 = w.i * Walk<D>::per_tile(p), r1 = min(w.q.n, r0 + Walk<D>::per_tile(p));
  const int past = w.q.len - w.q.n, first = past + r0 + 1, last = past + r1;
  *hi = first > 0 ? first / KB : 0;
  *lo = p.a.window > 0 && p.a.window < last ? (int)((uint32_t)(last - (int)p.a.window + KB - 1) / KB) : 0;
}

// NaN scales of the values that a row sees in this segment: a bit per 16 columns.  The products take such a scale as
// zero, since their other rows may not see it.  The V warps note the groups of columns that they met one in, in blocks
// that all of the tile's rows see; for a block at the border of some row they note only that, and the keys there are
// looked up in the pages again.  They lie within the tile's rows and two blocks of either border: some hundreds, however
// long the sequence is, so that no other role's wait runs out meanwhile.
template <int D>
__device__ __noinline__ uint32_t nan_columns(const TileParams& p, const TileShared& sh, const Walk<D>& w, int row_lo, int row_hi) {
  constexpr int KB = TileCfg<D>::kKeys;
  const volatile int* what = sh.nan_what[w.no & 7];
  uint32_t bits = 0;
  for (int s = 0; s < D / 16; ++s)
    if (what[s] == w.no + 1) bits |= 1u << s;
  if (what[kNanAtBorder] != w.no + 1) return bits;
  const AttendLaunch& a = p.a;
  int lo, hi;
  seen_by_all(p, w, &lo, &hi);
  const int64_t k0 = max((int64_t)row_lo, (int64_t)(w.first + w.at) * KB);
  const int64_t k1 = min((int64_t)row_hi, (int64_t)(w.first + w.end) * KB);
  for (int64_t j = k0; j < k1; ++j) {
    if (j >= (int64_t)lo * KB && j < (int64_t)hi * KB) {
      j = (int64_t)hi * KB - 1;
      continue;
    }
    const int page = __ldg(a.tables + w.b * a.ldt + (j >> a.cache.page_shift));
    if (page < 0 || page >= a.cache.pages) continue;
    const int in = (int)j & (a.cache.page_size - 1);
    const uint8_t* tile = kv_tile<D>(a.cache, page, w.h, in);
    for (int s = 0; s < D / 16; ++s)
      if ((tile[kv_v_scale(D, in % kKvTile, s)] & 0x7F) == 0x7F) bits |= 1u << s;
  }
  return bits;
}

// Tile holding key k of a sequence, on page `page` (page 0 if that is none).
template <int D>
__device__ __forceinline__ const uint8_t* tile_at(const KvCache& c, int page, int h, int k) {
  const uint32_t pg = page >= 0 && page < c.pages ? page : 0;
  const uint32_t stride = (uint32_t)(c.page_stride >> 7), tiles = (uint32_t)c.page_size / kKvTile;
  return c.data + (((uint64_t)pg * stride) << 7) +
         (h * tiles + (((uint32_t)k & (c.page_size - 1)) / kKvTile)) * (uint64_t)kv_tile_bytes(D);
}

template <int D>
__global__ void __launch_bounds__(TileCfg<D>::kThreads, 1) k_attend_tile(const TileParams p) {
  using C = TileCfg<D>;
  constexpr int KB = C::kKeys, SB = C::kSBufs, W = C::kThreads / 32;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_u = smem_u32(smem_raw), base = (raw_u + 1023u) & ~1023u;
  TileShared& sh = *reinterpret_cast<TileShared*>(smem_raw + (base - raw_u) + C::kOffMeta);
  const uint32_t sQ = base, sK = base + C::kOffK, sV = base + C::kOffV;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  volatile int* abort = &sh.abort;
  const uint32_t bar0 = smem_u32(sh.bars);
  const uint32_t q_full = bar0, k_full = q_full + 16, k_empty = k_full + 16, v_full = k_empty + 16, v_empty = v_full + 16;
  const uint32_t s_full = v_empty + 16;                  // [row tile or buffer]
  const uint32_t p_full = s_full + 16, pv_done = p_full + 16, joined = pv_done + 16, told = joined + 8;
  const uint32_t half_full = told + 8, half_read = half_full + 8, drain = half_read + 8, p_half = drain + 8;

  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(q_full + 8 * i, 4);
      mbar_init(k_full + 8 * i, 4);
      mbar_init(k_empty + 8 * i, 1);
      mbar_init(v_full + 8 * i, C::kVWarps);
      mbar_init(v_empty + 8 * i, 1);
      mbar_init(s_full + 8 * i, 1);
      mbar_init(p_full + 8 * i, 4);
      mbar_init(p_half + 8 * i, 4);
      mbar_init(pv_done + 8 * i, 1);
    }
    mbar_init(joined, C::kSoftWarps);
    mbar_init(told, 1);
    mbar_init(half_full, 4);
    mbar_init(half_read, 4);
    mbar_init(drain, 1);
    sh.abort = 0;
    for (int i = 0; i < 8; ++i) {
      sh.nan_seg[i] = 0;
      for (int k = 0; k <= kNanAtBorder; ++k) sh.nan_what[i][k] = 0;
    }
  }
  if (warp == C::kWarpMma) tmem_alloc(smem_u32(&sh.tmem), 512);
  fence_mbar_init();

  // ---- the line: twice over the tiles, for their units' number and for this CTA's first
  const int per_tile = p.tokens * C::kRowTiles, Hkv = p.a.cache.heads;
  int64_t total = 0, cta0 = 0, cta1 = 0, G = 0;
  for (int pass = 0; pass < 2; ++pass) {
    int64_t done = 0;
    for (int64_t b0 = 0; b0 < p.a.B; b0 += C::kThreads) {
      const int64_t b = b0 + tid;
      int64_t tiles = 0, round;
      if (b < p.a.B) tiles = (tile_seq(p.a, b).n + per_tile - 1) / per_tile;
      const int64_t mine = block_prefix<W>(tiles, sh.scan, &round);
      sh.seq_first[tid] = mine;
      if (tid == 0) sh.seq_first[C::kThreads] = round;
      __syncthreads();
      for (int64_t f0 = 0; f0 < round; f0 += C::kThreads) {
        const int64_t f = f0 + tid;
        int count = 0, first, at = 0, i = 0;
        AttendSeq q = {};
        if (f < round) {
          int hi = C::kThreads;  // the last sequence of the round whose first tile is at or before f
          while (hi - at > 1) {
            const int mid = (at + hi) >> 1;
            if (sh.seq_first[mid] <= f) at = mid;
            else hi = mid;
          }
          i = (int)(f - sh.seq_first[at]);
          q = tile_seq(p.a, b0 + at);
          tile_blocks<D>(p.a, q, i, per_tile, &first, &count);
          if (pass == 0 && count == 0 && f % gridDim.x == blockIdx.x) {  // no key: its rows are zeros
            const int r1 = min(q.n, (i + 1) * per_tile);
            for (int r = i * per_tile; r < r1; ++r) {
              uint4* row = reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(p.a.out) + (int64_t)(q.s0 + r) * p.a.ldo);
              for (int e = 0; e < p.a.q_heads * D / 8; ++e) row[e] = make_uint4(0, 0, 0, 0);
            }
          }
        }
        int64_t all;
        const int units = count ? count + kLead : 0;
        const int64_t before = (done + block_prefix<W>(units, sh.scan, &all)) * Hkv;
        if (pass == 1 && cta0 >= before && cta0 < before + (int64_t)units * Hkv) {
          sh.b = (int)(b0 + at);
          sh.i = i;
          sh.before = before;
        }
        done += all;
      }
      __syncthreads();
    }
    if (pass == 0) {
      total = done * Hkv;
      G = min((int64_t)p.G, total);
      if (blockIdx.x < G) {
        cta0 = blockIdx.x * total / G;
        cta1 = (blockIdx.x + 1) * total / G;
      } else {
        break;
      }
    }
  }
  if (tid == 0) {
    sh.G = G;
    sh.total = total;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  bool ok = true;

  if (cta0 < cta1) {
    if (warp < C::kSoftWarps) {
      // ------------------------------------------------------------ softmax
      const int X = warp >> 2, r = tid & 127;           // row tile, row of it
      const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
      const uint32_t tO = tmem + lanes + C::kTmemO + X * D;
      const uint32_t qwarp = sQ + X * C::kQBytes + (warp & 3) * 4096;  // this warp's 32 rows
      constexpr int LR = D / 8, RI = 32 / LR;           // lanes a row takes, rows a load takes
      // the walk stays in shared memory: the block loop needs the registers
      static_assert(sizeof(Walk<D>) <= 96, "a warp's walk");
      Walk<D>& w = *reinterpret_cast<Walk<D>*>(sh.walk + warp * 96);
      int more = 0;
      if (lane == 0) more = w.start(p, sh, cta0, cta1);
      more = __shfl_sync(0xffffffffu, more, 0);
      // Phases and flags in one register: bits 0, 1 the score buffers, 2 P V done, 3 halves joined, 4 parts
      // joined, 5 some key seen, 6 a block before this one in the segment.  What else the block loop
      // does not need in registers is in shared memory (a spill would go through an L1 of a few KB).
      constexpr uint32_t kPv = 4, kHalf = 8, kPart = 16, kAny = 32, kLater = 64;
      uint32_t st = 0;
      const uint32_t row_at = smem_u32(sh.row[tid]);
      while (more) {
        __syncwarp();
        const bool halved = w.halved(p);
        // blocks from `b0` on, every `step`-th; the second half of one block is empty
        const int b0 = w.at + (halved ? X : 0);
        const bool mine_seg = b0 < w.end;
        const int XR = halved ? 0 : X;                  // whose rows
        const int tok = p.a.group == 1 ? r : __umulhi(r, p.by_group), inner = r - tok * p.a.group;
        const int idx = w.i * per_tile + XR * p.tokens + tok;
        const bool live = mine_seg && tok < p.tokens && idx < w.q.n;
        auto at_row = [&](int64_t ld) {                 // of q or out, in elements
          const int row = halved ? 0 : X;
          return (int64_t)(w.q.s0 + w.i * per_tile + row * p.tokens + tok) * ld + (int64_t)(w.h * p.a.group + inner) * D;
        };
        const int seen = w.q.len - w.q.n + idx + 1;       // keys up to the row's own
        // keys [row_lo, row_hi) are those that the row sees
        const int row_hi = live ? max(seen, 0) : 0x7FFFFFFF;
        const int row_lo = live && p.a.window > 0 && p.a.window < row_hi ? row_hi - (int)p.a.window : 0;
        float m = -INFINITY, l = 0.0f;
        st &= ~(kAny | kLater);
        if (mine_seg) {
          // ---- Q
          // LR lanes take a row 16 bytes each, so that a load meets few lines; a lane keeps the power of
          // two of its own row
          const float unit = p.a.scale * kLog2e * p.a.cache.k_scale[w.h];
          const uint32_t sign = unit < 0.0f ? 0x80008000u : 0u;  // a negative scale goes into q: the largest product is the largest score
          const int64_t from = live ? at_row(p.a.ldq) : -1;
          const float value_scale = __ldg(p.a.cache.v_scale + w.h);
          const float sink = live && p.a.sinks ? __ldg(p.a.sinks + w.h * p.a.group + inner) : -INFINITY;
          int pw = 0;
#pragma unroll 1
          for (int i0 = 0; i0 < 32; i0 += 8 * RI) {
            uint4 v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int64_t f = __shfl_sync(0xffffffffu, from, i0 + i * RI + lane / LR);
              v[i] = make_uint4(0, 0, 0, 0);
              if (f >= 0) v[i] = *reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(p.a.q) + f + (lane % LR) * 8);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              int mx = act_maxmag8(reinterpret_cast<const uint32_t*>(&v[i]));
#pragma unroll
              for (int k = 1; k < LR; k <<= 1) mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, k));
              const int pr = act_pow2(mx), row = i0 + i * RI + lane / LR, c = lane % LR;
              const int mine = __shfl_sync(0xffffffffu, pr, (lane % RI) * LR);
              if (lane / RI == i0 / RI + i) pw = mine;
              const uint4 f = act_granule_f16(reinterpret_cast<const uint32_t*>(&v[i]), pr);
              st_shared_v4(qwarp + (c >> 3) * 16384 + row * 128 + (((c & 7) ^ (row & 7)) << 4), f.x ^ sign, f.y ^ sign, f.z ^ sign, f.w ^ sign);
            }
          }
          float factor = fabsf(unit) * pow2f(pw);
          if (factor == 0.0f) factor = 1e-38f;  // every score 0, a masked one (-inf) stays out
          st_shared_v4(row_at, row_lo, row_hi, __float_as_uint(factor), __float_as_uint(sink));
          if (lane == 0) sh.value[warp] = value_scale;
          fence_proxy_async_smem();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(q_full + 8 * X);
          const bool idle = !__any_sync(0xffffffffu, live);  // no row of this warp counts
          // pages of the block's tiles that are not there, a block ahead
          auto pages_of = [&](int blk) -> bool {
            if (lane >= KB / 16) return true;
            const int k = (w.first + blk) * KB + lane * 16;
            if (k >= w.q.len) return true;
            const int page = __ldg(p.a.tables + w.b * p.a.ldt + (k >> p.a.cache.page_shift));
            return page >= 0 && page < p.a.cache.pages;
          };
          bool page_ok = pages_of(b0);
#pragma unroll 1
          for (int blk = b0; blk < w.end; blk += halved ? 2 : 1) {
            const uint32_t sbuf = SB == 2 ? (blk - w.at) & 1 : X;
            const uint32_t tS = tmem + lanes + sbuf * KB;
            const uint32_t gone = ~__ballot_sync(0xffffffffu, page_ok) & ((1u << (KB / 16)) - 1);
            if (blk + (halved ? 2 : 1) < w.end) page_ok = pages_of(blk + (halved ? 2 : 1));
            const int k0 = (w.first + blk) * KB;
            // columns [lo, hi) that the row sees
            const uint2 sees = ld_shared_v2(row_at);
            const int hi = min(KB, max((int)sees.y - k0, 0));
            const int lo = min(KB, max((int)sees.x - k0, 0));
            const bool edge = __any_sync(0xffffffffu, hi < KB || lo > 0) || gone;
            if (!(ok = warp_wait(s_full + 8 * sbuf, (st >> sbuf) & 1, abort, p.wait_ns))) break;
            st ^= 1u << sbuf;
            tc_fence_after();
            if (!idle) {
              uint32_t v[2][32];
              if (edge) {  // scores that a row does not see become -inf in their place
#pragma unroll 1
                for (int c = 0; c < KB; c += 32) {
                  // columns of these 32 that the row sees, a bit each
                  uint32_t seen = hi - c >= 32 ? 0xFFFFFFFFu : hi <= c ? 0u : (1u << (hi - c)) - 1;
                  if (lo > c) seen &= lo - c >= 32 ? 0u : 0xFFFFFFFFu << (lo - c);
                  if ((gone >> (c >> 4)) & 1) seen &= 0xFFFF0000u;
                  if ((gone >> (c >> 4)) & 2) seen &= 0x0000FFFFu;
                  if (__all_sync(0xffffffffu, seen == 0xFFFFFFFFu)) continue;
                  tmem_ld32(tS + c, v[0]);
#pragma unroll
                  for (int e = 0; e < 32; ++e)
                    if (!((seen >> e) & 1)) v[0][e] = 0xFF800000u;
                  tmem_st32(tS + c, v[0]);
                }
                tmem_st_wait();
                bool some = lo < hi;
                if (gone) {
                  some = false;
                  for (int g = 0; g < KB / 16; ++g)
                    some |= !((gone >> g) & 1) && max(lo, g * 16) < min(hi, g * 16 + 16);
                }
                if (some) st |= kAny;
              } else {
                st |= kAny;
              }
              // the maximum; the last 64 scores stay in registers.  Every load waits in its own statement: a load under
              // way writes its registers when it likes, and this loop has branches and loop edges that may move them
              // (8192 rows, 32 heads on 4 of 128: loads issued ahead of their wait took 552 us, these 536).
              float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
              for (int c = 0; c < KB; c += 64) {
                tmem_ld32(tS + c, v[0]);
                tmem_ld32(tS + c + 32, v[1]);
#pragma unroll
                for (int e = 0; e < 32; e += 4) {
#pragma unroll
                  for (int k = 0; k < 2; ++k) {
                    top[2 * k] = max3(top[2 * k], __uint_as_float(v[k][e]), __uint_as_float(v[k][e + 1]));
                    top[2 * k + 1] = max3(top[2 * k + 1], __uint_as_float(v[k][e + 2]), __uint_as_float(v[k][e + 3]));
                  }
                }
              }
              const float best = fmaxf(max3(top[0], top[1], top[2]), top[3]);
              const float mul = __uint_as_float(ld_shared_v2(row_at + 8).x);
              const float mx = best == -INFINITY ? best : best * mul;
              const float mn = (m == -INFINITY || mx > m + kSlack) ? fmaxf(m, mx) : m;
              if ((st & kLater) && __any_sync(0xffffffffu, mn > m)) {
                if (!(ok = warp_wait(pv_done + 8 * X, !(st & kPv), abort, p.wait_ns))) break;
                tc_fence_after();
                const float f = mn > m ? fast_exp2(m - mn) : 1.0f;
                l *= f;
#pragma unroll 1
                for (int c = 0; c < D; c += 16) {
                  uint32_t o[16];
                  tmem_ld16(tO + c, o);
#pragma unroll
                  for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                  tmem_st16(tO + c, o);
                }
              }
              m = mn;
              const float off = kPBias - (m == -INFINITY ? 0.0f : m);
              const uint64_t mul2 = pair(mul, mul), off2 = pair(off, off);
              uint64_t sum[2] = {0, 0};
              // P, two f16 a column, over the second half of the scores: those are in registers
              auto probabilities = [&](const uint32_t (&x)[32], int c) {
#pragma unroll
                for (int h = 0; h < 32; h += 16) {
                  uint32_t pk[8];
#pragma unroll
                  for (int e = 0; e < 16; e += 2) {
                    float a, b;
                    split(fma2(pair(__uint_as_float(x[h + e]), __uint_as_float(x[h + e + 1])), mul2, off2), a, b);
                    a = fast_exp2(a);
                    b = fast_exp2(b);
                    sum[(e >> 1) & 1] = add2(sum[(e >> 1) & 1], pair(a, b));
                    pk[e >> 1] = pack_half2(a, b);
                  }
                  tmem_st8(tS + KB / 2 + (c + h) / 2, pk);
                }
              };
#pragma unroll 1
              for (int c = KB - 64;; c -= 64) {
                probabilities(v[0], c);
                if (c) tmem_ld32(tS, v[0]);
                probabilities(v[1], c + 32);
                if (!c) break;
                // the second half's products may begin
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(p_half + 8 * sbuf);
                __syncwarp();
                tmem_ld32(tS + 32, v[1]);
              }
              float la, lb;
              split(add2(sum[0], sum[1]), la, lb);
              l += la + lb;
              tmem_st_wait();
            } else if (KB == 128) {
              if (lane == 0) mbar_arrive(p_half + 8 * sbuf);
            }
            // With two score buffers this block's scores do not say that the last block's P V is done.  It is
            // waited for here, one phase at a time: a wait on a phase takes the one before it for done.
            if (SB == 2 && (st & kLater) && !(ok = warp_wait(pv_done + 8 * X, !(st & kPv), abort, p.wait_ns))) break;
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(p_full + 8 * sbuf);
            st = (st ^ kPv) | kLater;
          }
          if (!ok) break;
          if (!(ok = warp_wait(pv_done + 8 * X, !(st & kPv), abort, p.wait_ns))) break;
          tc_fence_after();
        }
        // ---- the two halves of a single row tile: the second's sums to the first
        const bool other = halved && w.end - w.at > 1;
        bool any = st & kAny;
        float f0 = 1.0f, f1 = 0.0f;
        if (other) {
          if (X == 1) {
            sh.half_m[r] = m;
            sh.half_l[r] = l;
            sh.half_any[r] = any;
            __syncwarp();
            if (lane == 0) mbar_arrive(half_full);
            if (!(ok = warp_wait(half_read, (st & kHalf) != 0, abort, p.wait_ns))) break;
          } else {
            if (!(ok = warp_wait(half_full, (st & kHalf) != 0, abort, p.wait_ns))) break;
            tc_fence_after();
            const float m1 = sh.half_m[r], mt = fmaxf(m, m1), ms = mt == -INFINITY ? 0.0f : mt;
            f0 = fast_exp2(m - ms);
            f1 = fast_exp2(m1 - ms);
            l = l * f0 + sh.half_l[r] * f1;
            any |= sh.half_any[r] != 0;
            m = mt;
          }
          st ^= kHalf;
        }
        const bool out = mine_seg && !(halved && X == 1);
        const bool whole = w.whole();
        auto sink_of = [&]() { return __uint_as_float(ld_shared_v2(row_at + 8).y); };
        float* part = p.parts + ((int64_t)blockIdx.x * 2 + (w.at == 0)) * C::kPartFloats;
        uint32_t lost = 0;
        if (live && out && *reinterpret_cast<volatile int*>(&sh.nan_seg[w.no & 7]) == w.no + 1)
          lost = nan_columns<D>(p, sh, w, row_lo, row_hi);
        __syncwarp();  // lanes come back from that one by one; the loads from TMEM take the whole warp
        auto value = [&](uint32_t v, int col) {
          return (lost >> (col >> 4)) & 1 ? __uint_as_float(0x7FC00000u) : __uint_as_float(v);
        };
        if (out) {
          const float f = whole && live && any ? out_factor(sh.value[warp], sink_of(), m, l, kPBias) : 0.0f;
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {
            uint32_t v[32];
            tmem_ld32(tO + c * 32, v);
            if (other) {
              uint32_t u[32];
              tmem_ld32(tO + D + c * 32, u);
#pragma unroll
              for (int e = 0; e < 32; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * f0 + __uint_as_float(u[e]) * f1);
            }
            if (whole) {  // to the place of Q, whose products are done
#pragma unroll
              for (int e = 0; e < 32; e += 8) {
                uint32_t o[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                  const int col = c * 32 + e + 2 * k;
                  const float x = any ? value(v[e + 2 * k], col) * f : 0.0f, y = any ? value(v[e + 2 * k + 1], col) * f : 0.0f;
                  const __nv_bfloat162 h2 = __floats2bfloat162_rn(x, y);
                  o[k] = *reinterpret_cast<const uint32_t*>(&h2);
                }
                const int chunk = c * 4 + e / 8;
                st_shared_v4(qwarp + (chunk >> 3) * 16384 + lane * 128 + (((chunk & 7) ^ (lane & 7)) << 4), o[0], o[1], o[2], o[3]);
              }
            } else if (live) {
#pragma unroll
              for (int e = 0; e < 32; e += 4) {
                const int col = c * 32 + e;
                __stcg(reinterpret_cast<float4*>(part) + (int64_t)(col / 4) * C::kRows + X * 128 + r,
                       make_float4(value(v[e], col), value(v[e + 1], col), value(v[e + 2], col), value(v[e + 3], col)));
              }
            }
            __syncwarp();  // the next load from TMEM takes the whole warp
          }
          if (other) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(half_read);
          }
          if (whole) {
            const int64_t to = live ? at_row(p.a.ldo) : -1;
#pragma unroll 4
            for (int i = 0; i < 32; i += RI) {
              const int row = i + lane / LR, c = lane % LR;
              const int64_t at = __shfl_sync(0xffffffffu, to, row);
              const int4 o = ld_shared_v4(qwarp + (c >> 3) * 16384 + row * 128 + (((c & 7) ^ (row & 7)) << 4));
              if (at >= 0) *reinterpret_cast<int4*>(reinterpret_cast<__nv_bfloat16*>(p.a.out) + at + c * 8) = o;
            }
            __syncwarp();
          }
          if (live && !whole) {
            float* st = part + C::kRows * D + X * 128 + r;
            __stcg(st, m);
            __stcg(st + C::kRows, l);
            __stcg(st + 2 * C::kRows, any ? 1.0f : 0.0f);
          }
        }
        if (!whole) {
          // ---- a part: the last of the tile's CTAs joins them, in the order of the line
          const int64_t seg1 = w.seg0 + w.count;
          const int64_t total_units = *reinterpret_cast<volatile int64_t*>(&sh.total), ctas = *reinterpret_cast<volatile int64_t*>(&sh.G);
          const int64_t c0 = ((w.seg0 + 1) * ctas - 1) / total_units, c1 = (seg1 * ctas - 1) / total_units;
          __syncwarp();
          if (lane == 0) mbar_arrive(joined);  // (the fence below covers what these warps wrote before)
          if (warp == 0) {
            if (!(ok = warp_wait(joined, (st & kPart) != 0, abort, p.wait_ns))) break;
            if (lane == 0) {
              uint32_t* count = reinterpret_cast<uint32_t*>(p.a.workspace + kTileCounts) + c0;
              __threadfence();
              const bool last = atomicAdd(count, 1u) == (uint32_t)(c1 - c0);
              if (last) *count = 0;  // for the next call
              __threadfence();
              *reinterpret_cast<volatile int*>(&sh.last) = last;
              mbar_arrive(told);
            }
            __syncwarp();
          }
          if (!(ok = warp_wait(told, (st & kPart) != 0, abort, p.wait_ns))) break;
          st ^= kPart;
          if (*reinterpret_cast<volatile int*>(&sh.last)) {
            const int n = (int)(c1 - c0) + 1;
            // CTA c0's part is in its slot 1, the others' in their slot 0
            auto part_of = [&](int k) { return p.parts + (2 * (c0 + k) + (k == 0)) * (int64_t)C::kPartFloats; };
            if (live && out) {
              float mt = -INFINITY, lt = 0.0f;
              bool at = false;
              for (int k = 0; k < n; ++k) {
                const float* st = part_of(k) + C::kRows * D + X * 128 + r;
                mt = fmaxf(mt, __ldcg(st));
                at |= __ldcg(st + 2 * C::kRows) != 0.0f;
              }
              const float ms = mt == -INFINITY ? 0.0f : mt;
              for (int k = 0; k < n; ++k) {
                const float* st = part_of(k) + C::kRows * D + X * 128 + r;
                lt += fast_exp2(__ldcg(st) - ms) * __ldcg(st + C::kRows);
              }
              const float f = at ? out_factor(sh.value[warp], sink_of(), mt, lt, kPBias) : 0.0f;
              __nv_bfloat16* dst = reinterpret_cast<__nv_bfloat16*>(p.a.out) + at_row(p.a.ldo);
#pragma unroll 1
              for (int c = 0; c < D / 16; ++c) {
                float4 o[4] = {};
                for (int k = 0; k < n; ++k) {
                  const float* q = part_of(k);
                  const float wk = fast_exp2(__ldcg(q + C::kRows * D + X * 128 + r) - ms);
#pragma unroll
                  for (int e = 0; e < 4; ++e) {
                    const float4 v = __ldcg(reinterpret_cast<const float4*>(q) + (int64_t)(c * 4 + e) * C::kRows + X * 128 + r);
                    o[e].x += wk * v.x, o[e].y += wk * v.y, o[e].z += wk * v.z, o[e].w += wk * v.w;
                  }
                }
#pragma unroll
                for (int e = 0; e < 4; e += 2) {
                  float x[8] = {o[e].x, o[e].y, o[e].z, o[e].w, o[e + 1].x, o[e + 1].y, o[e + 1].z, o[e + 1].w};
                  uint32_t b[4];
#pragma unroll
                  for (int k = 0; k < 4; ++k) {
                    const __nv_bfloat162 h2 = __floats2bfloat162_rn(at ? x[2 * k] * f : 0.0f, at ? x[2 * k + 1] * f : 0.0f);
                    b[k] = *reinterpret_cast<const uint32_t*>(&h2);
                  }
                  *reinterpret_cast<uint4*>(dst + c * 16 + e * 4) = make_uint4(b[0], b[1], b[2], b[3]);
                }
              }
            }
          }
        }
        __syncwarp();
        if (lane == 0) more = w.next(p);
        more = __shfl_sync(0xffffffffu, more, 0);
      }
    } else if (warp < C::kWarpV) {
      // ------------------------------------------------------------ K to f16
      const int kw = warp - C::kWarpK, mu = lane & 15, half = lane >> 4;
      const int tok = kv_mma_token(mu);
      // the lane's codes and scales in a tile: 64 values of row mu
      const int at = D == 64 ? mu * 32 : mu * 64 + half * 32;
      const int sat = 8 * D + (D == 64 ? (mu & 7) * 8 : (mu & 7) * 16 + half * 8) - at;
      uint4 code[C::kKJobs][2];
      uint2 sc[C::kKJobs];
      // the tile (of 16 tokens) of job j and this lane, counted in the block
      auto tile_of = [&](int j) { return D == 64 ? 2 * kw + half : D == 128 ? kw + 4 * j : kw; };
      Walk<D> ld;
      bool more = ld.start(p, sh, cta0, cta1), pending = false;  // a block to load; one loaded
      int lblk = ld.at;
      int page[C::kKJobs];
      auto fetch = [&]() {  // pages of the block to be loaded next
#pragma unroll
        for (int j = 0; j < C::kKJobs; ++j) {
          const int k = (ld.first + lblk) * KB + tile_of(j) * 16;
          page[j] = k < ld.q.len ? __ldg(p.a.tables + ld.b * p.a.ldt + (k >> p.a.cache.page_shift)) : -1;
        }
      };
      auto load = [&]() {
#pragma unroll
        for (int j = 0; j < C::kKJobs; ++j) {
          // (a page that is not there: page 0's, whose scores are masked)
          const uint8_t* tile = tile_at<D>(p.a.cache, page[j], ld.h, (ld.first + lblk) * KB + tile_of(j) * 16) +
                                (D == 256 ? j * 1024 : 0) + at;
          code[j][0] = *reinterpret_cast<const uint4*>(tile);
          code[j][1] = *reinterpret_cast<const uint4*>(tile + 16);
          sc[j] = *reinterpret_cast<const uint2*>(tile + (D == 256 ? j * (128 - 1024) : 0) + sat);
        }
        if (++lblk == ld.end) {
          more = ld.next(p);
          lblk = ld.at;
        }
        if (more) fetch();
      };
      if (more) fetch();
      uint32_t it = 0;
      bool stopped = false;
      auto step = [&]() -> bool {
        if (it == p.hold) {
          if (!p.pause) {
            stopped = true;
            return false;
          }
          pause();
        }
        const uint32_t stage = it & 1;
        if (!warp_wait(k_empty + 8 * stage, ((it >> 1) & 1) ^ 1, abort, p.wait_ns)) return false;
#pragma unroll
        for (int j = 0; j < C::kKJobs; ++j) {
          const uint32_t s4 = D == 64 ? __byte_perm(sc[j].x, sc[j].y, mu >> 3 ? 0x7531 : 0x6420)
                                      : __byte_perm(sc[j].x, sc[j].y, mu >> 3 ? 0x7632 : 0x5410);
          const uint32_t s01 = e4m3x2_to_f16x2(s4), s23 = e4m3x2_to_f16x2(s4 >> 16);
          const uint32_t s[4] = {bcast_lo(s01), bcast_hi(s01), bcast_lo(s23), bcast_hi(s23)};
          const int n = tile_of(j) * 16 + tok, sub = D == 64 ? 0 : D == 128 ? half : 2 * j + half;
          const uint32_t row = sK + stage * C::kKvBytes + sub * (KB * 128) + n * 128;
          const uint32_t wd[8] = {code[j][0].x, code[j][0].y, code[j][0].z, code[j][0].w,
                                  code[j][1].x, code[j][1].y, code[j][1].z, code[j][1].w};
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            uint32_t f[4];
            e2m1x8_to_f16x8(wd[c], f[0], f[1], f[2], f[3]);
#pragma unroll
            for (int e = 0; e < 4; ++e) f[e] = hmul2_u32(f[e], s[c >> 1]);
            st_shared_v4(row + ((c ^ (n & 7)) << 4), f[0], f[1], f[2], f[3]);
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(k_full + 8 * stage);
        ++it;
        return true;
      };
      while ((!pending || (ok = step())) && more) {
        load();  // in flight while the stages are full
        pending = true;
      }
      ok |= stopped;  // (no wait of this warp's ran out)
    } else if (warp < C::kWarpMma) {
      // ------------------------------------------------------------ V to f16, turned
      const int vw = warp - C::kWarpV;
      const int half = D == 64 ? (lane >> 3) & 1 : lane >> 4, o = D == 64 ? lane & 7 : lane & 15;
      // the lane's codes in a tile: 8 columns of tokens 8 half + i; their scales
      const int at0 = 9 * D + (D == 64 ? half * 256 : half * 512) + o * 4, at1 = 9 * D + half * 512 + ((o * 4) ^ 32);
      const int sat = 17 * D + (o >> 1) * 16;
      uint32_t code[C::kVJobs][8];
      uint4 sc[C::kVJobs];
      int nvalid[C::kVJobs];   // of the lane's 8 tokens
      int segno;
      // job vw + j * kVWarps: its tile (of 16 tokens) and, at head_dim 256, column block
      auto job_of = [&](int j) { return vw + j * C::kVWarps; };
      auto tile_of = [&](int j) { return D == 64 ? 2 * job_of(j) + (lane >> 4) : D == 128 ? job_of(j) : job_of(j) & 3; };
      auto block_of = [&](int j) { return D == 256 ? job_of(j) >> 2 : 0; };
      Walk<D> ld;
      bool more = ld.start(p, sh, cta0, cta1), pending = false;  // a block to load; one loaded
      int lblk = ld.at;
      int page[C::kVJobs];
      uint32_t it = 0;
      // which of the segment's blocks, the first being the warp's n-th, every row sees: for the rare block that holds a NaN
      auto note = [&](uint32_t n) {
        int lo, hi;
        seen_by_all(p, ld, &lo, &hi);
        sh.v_seen[vw][ld.no & 1] = make_int2(n + lo - ld.first - ld.at, n + hi - ld.first - ld.at);
      };
      auto fetch = [&]() {
#pragma unroll
        for (int j = 0; j < C::kVJobs; ++j) {
          const int k = (ld.first + lblk) * KB + tile_of(j) * 16;
          page[j] = job_of(j) < C::kAllJobs && k < ld.q.len ? __ldg(p.a.tables + ld.b * p.a.ldt + (k >> p.a.cache.page_shift)) : -1;
        }
      };
      auto load = [&]() {
        segno = ld.no;
#pragma unroll
        for (int j = 0; j < C::kVJobs; ++j) {
          const int k = (ld.first + lblk) * KB + tile_of(j) * 16;
          // (a page that is not there: page 0's, with scales taken as zero)
          const uint8_t* tile = tile_at<D>(p.a.cache, page[j], ld.h, k) + block_of(j) * 1024;
#pragma unroll
          for (int i = 0; i < 8; ++i)
            code[j][i] = *reinterpret_cast<const uint32_t*>(tile + ((i & 2) && D > 64 ? at1 : at0) + i * (D == 64 ? 32 : 64));
          sc[j] = *reinterpret_cast<const uint4*>(tile + sat + block_of(j) * (128 - 1024));
          nvalid[j] = page[j] >= 0 && page[j] < p.a.cache.pages ? min(8, max(ld.q.len - k - 8 * half, 0)) : 0;
        }
        if (++lblk == ld.end) {
          more = ld.next(p);
          lblk = ld.at;
          if (more) note(it + 1);
        }
        if (more) fetch();
      };
      if (more) fetch(), note(0);
      const int rot = o & 3, odd = (o >> 2) & 1;
      uint32_t place[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int d0 = 2 * ((e + rot) & 3) + odd;
        place[e] = d0 * 128 + ((half ^ d0) << 4);
      }
      const uint32_t rsel = rot == 0 ? 0x3210 : rot == 1 ? 0x0321 : rot == 2 ? 0x1032 : 0x2103;
      auto step = [&]() -> bool {
        const uint32_t stage = it & 1;
        if (!warp_wait(v_empty + 8 * stage, ((it >> 1) & 1) ^ 1, abort, p.wait_ns)) return false;
        uint32_t met = 0;        // a NaN scale, a bit per column block
#pragma unroll
        for (int j = 0; j < C::kVJobs; ++j) {
          if (job_of(j) >= C::kAllJobs) break;
          // scales of the lane's tokens 0..3 and 4..7, a byte each
          const uint4 sw = sc[j];
          const uint32_t s0 = half ? 0x62 : 0x40, s1 = half ? 0x73 : 0x51;
          uint32_t q[2] = {__byte_perm(__byte_perm(sw.x, sw.y, s0), __byte_perm(sw.z, sw.w, s0), 0x5410),
                           __byte_perm(__byte_perm(sw.x, sw.y, s1), __byte_perm(sw.z, sw.w, s1), 0x5410)};
          const int nv = nvalid[j];
          if (nv < 8) {  // places behind the last key hold anything
            q[1] = nv > 4 ? q[1] & ((1u << (8 * (nv - 4))) - 1) : 0u;
            if (nv < 4) q[0] &= (1u << (8 * nv)) - 1;
          }
          const uint32_t nan0 = ((q[0] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
          const uint32_t nan1 = ((q[1] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
          if (nan0 | nan1) {
            q[0] &= ~((nan0 >> 7) * 0xFFu);
            q[1] &= ~((nan1 >> 7) * 0xFFu);
            met |= 1u << block_of(j);
          }
          uint32_t x[4][4], y[4][4];  // [d][pair of tokens]
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            constexpr uint32_t M = 0x0F0F0F0Fu;
            const uint32_t a = code[j][2 * i], b = code[j][2 * i + 1];
            const uint32_t even = __byte_perm((a & M) | ((b << 4) & ~M), 0, rsel);
            const uint32_t oddw = __byte_perm(((a >> 4) & M) | (b & ~M), 0, rsel);
            const uint32_t u = odd ? oddw : even, v = odd ? even : oddw;
            const uint32_t s = e4m3x2_to_f16x2(q[i >> 1] >> (16 * (i & 1)));
            uint32_t f[4], g[4];
            e2m1x8_to_f16x8(u, f[0], f[1], f[2], f[3]);
            e2m1x8_to_f16x8(v, g[0], g[1], g[2], g[3]);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              x[e][i] = hmul2_u32(f[e], s);
              y[e][i] = hmul2_u32(g[e], s);
            }
          }
          const int ti = tile_of(j);
          const uint32_t to = sV + stage * C::kKvBytes + (ti >> 2) * (D * 128) + block_of(j) * 16384 + o * 1024;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            // row d0 of the octet and its neighbour d0 ^ 1; 16-byte place (2 (ti & 3) + half) ^ row
            const uint32_t at = place[e] ^ ((ti & 3) << 5);
            st_shared_v4(to | at, x[e][0], x[e][1], x[e][2], x[e][3]);
            st_shared_v4(to | (at ^ (128 + 16)), y[e][0], y[e][1], y[e][2], y[e][3]);
          }
        }
        // (noted behind the jobs, once: see the code's size above)
        if (met) {
          const int2 seen = sh.v_seen[vw][segno & 1];
          const bool inside = (int)it >= seen.x && (int)it < seen.y;
          for (int c = 0; c < 2; ++c)
            if ((met >> c) & 1)
              *reinterpret_cast<volatile int*>(&sh.nan_what[segno & 7][inside ? (o >> 1) + 8 * c : kNanAtBorder]) = segno + 1;
          *reinterpret_cast<volatile int*>(&sh.nan_seg[segno & 7]) = segno + 1;
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(v_full + 8 * stage);
        ++it;
        return true;
      };
      while ((!pending || (ok = step())) && more) {
        load();
        pending = true;
      }
    } else {
      // ------------------------------------------------------------ the products
      if (elect_one()) {
        constexpr uint32_t ids = idesc_f16(KB), ido = idesc_f16(D);
        uint32_t it = 0, q_turn = 0, p_turn = 0;  // blocks before this segment; phases, a bit per row tile or buffer
        auto wait = [&](uint32_t bar, uint32_t parity) { return ok = ok && wait_for(bar, parity, abort, p.wait_ns); };
        Walk<D> w;
        for (bool more = w.start(p, sh, cta0, cta1); more && ok; more = w.next(p)) {
          // A task is the two products of one row tile with one block: (block, row tile) in turn, or
          // the blocks alone where there is one row tile.  Task t takes score buffer t & 1; its
          // scores are issued two tasks ahead of its P V, behind the P V that read the buffer last.
          const bool both = w.row_tiles(p) == 2, halved = w.halved(p);
          const int tasks = (w.end - w.at) << (both ? 1 : 0);
#pragma unroll 1
          for (int u = 0; u < tasks + 2 && ok; ++u) {
            if (u >= 2) {
              const int t = u - 2, blk = both ? t >> 1 : t;
              const uint32_t n = it + blk, sbuf = t & 1, X = C::kRowTiles == 2 ? sbuf : 0;
              if (!wait((KB == 128 ? p_half : p_full) + 8 * sbuf, (p_turn >> sbuf) & 1)) break;
              if (!(both && sbuf) && !wait(v_full + 8 * (n & 1), (n >> 1) & 1)) break;
              tc_fence_after();
              uint32_t add = blk > (halved ? 1 : 0);
              const uint64_t vd = desc_sw128(sV + (n & 1) * C::kKvBytes);
              const uint32_t pt = tmem + sbuf * KB + KB / 2;
#pragma unroll 1
              for (int c = KB / 64 - 1; c >= 0; --c) {  // the keys whose probabilities come first
                if (KB == 128 && c == 0) {
                  if (!wait(p_full + 8 * sbuf, (p_turn >> sbuf) & 1)) break;
                  tc_fence_after();
                }
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) {
                  mma_f16_ta(tmem + C::kTmemO + X * D, pt + (c * 4 + kk) * 8, vd + c * (D * 8) + 2 * kk, ido, add);
                  add = 1;
                }
              }
              if (!ok) break;
              p_turn ^= 1u << sbuf;
              mma_commit(pv_done + 8 * X);
              if (!both || sbuf) mma_commit(v_empty + 8 * (n & 1));
            }
            if (u < tasks) {
              const uint32_t n = it + (both ? u >> 1 : u), sbuf = u & 1, X = both || halved ? sbuf : 0;
              if (!(both && sbuf) && !wait(k_full + 8 * (n & 1), (n >> 1) & 1)) break;
              if (u < (both || halved ? 2 : 1)) {
                if (!wait(q_full + 8 * X, (q_turn >> X) & 1)) break;
                q_turn ^= 1u << X;
              }
              tc_fence_after();
              const uint64_t qd = desc_sw128(sQ + X * C::kQBytes), kd = desc_sw128(sK + (n & 1) * C::kKvBytes);
              uint32_t add = 0;
#pragma unroll 1
              for (int c = 0; c < D / 64; ++c) {
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) {
                  mma_f16(tmem + sbuf * KB, qd + c * 1024 + 2 * kk, kd + c * (KB * 8) + 2 * kk, ids, add);
                  add = 1;
                }
              }
              mma_commit(s_full + 8 * sbuf);
              if (!both || sbuf) mma_commit(k_empty + 8 * (n & 1));
            }
          }
          it += w.end - w.at;
        }
        // every product issued has completed once this arrives
        mma_commit(drain);
        const uint64_t t0 = globaltimer_ns();
        while (!mbar_try_wait(drain, 0) && globaltimer_ns() - t0 < kWaitNs) {}
      }
    }
    if (!ok && (lane == 0 || warp == C::kWarpMma)) atomicExch(reinterpret_cast<int*>(p.a.workspace), 5);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  __syncwarp();
  if (warp == C::kWarpMma) tmem_dealloc(tmem, 512);
  pdl_wait();  // what follows this kernel in the stream follows the row kernel, too
}

template <int D>
cudaError_t go(TileParams p, cudaStream_t s) {
  using C = TileCfg<D>;
  static int done[64];
  constexpr size_t bytes = C::kOffMeta + sizeof(TileShared) + 1024;
  static_assert(bytes <= 232448, "shared memory");
  if (cudaError_t e = set_up_kernel(k_attend_tile<D>, bytes, done)) return e;
  // The two kernels of a call share neither rows nor workspace: this one starts on the SMs that the
  // row kernel leaves.  It is launched once every CTA of that one runs, so it may wait for its end.
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)p.G);
  cfg.blockDim = dim3((unsigned)C::kThreads);
  cfg.dynamicSmemBytes = bytes;
  cfg.stream = s;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_attend_tile<D>, p);
}

}  // namespace

size_t attend_tile_parts_bytes(int head_dim) {
  const size_t f = head_dim == 64 ? TileCfg<64>::kPartFloats : head_dim == 128 ? TileCfg<128>::kPartFloats : TileCfg<256>::kPartFloats;
  return 2 * (size_t)kMaxAttendGrid * f * 4;
}

cudaError_t launch_attend_tile(const AttendLaunch& L, int head_dim, cudaStream_t s) {
  TileParams p;
  p.a = L;
  p.G = sm_count() < kMaxAttendGrid ? sm_count() : kMaxAttendGrid;
  p.tokens = 128 / L.group;
  p.by_group = (uint32_t)(((uint64_t)1 << 32) / L.group + 1);
  p.parts = reinterpret_cast<float*>(L.workspace + kAttendCleared + attend_row_parts_bytes(head_dim));
  p.wait_ns = L.wait_ns ? L.wait_ns : kWaitNs;
  p.hold = L.withhold == 0 ? kNoHold : L.withhold > 0 ? L.withhold - 1 : -1 - L.withhold;
  p.pause = L.withhold < 0;
  return head_dim == 64 ? go<64>(p, s) : head_dim == 128 ? go<128>(p, s) : go<256>(p, s);
}

}  // namespace vt
