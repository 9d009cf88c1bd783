// Attention of few rows per sequence over the paged NVFP4 cache (the decode step, drafted tokens).
//
//   S^T = K Q^T,  p = 2^(s - m),  O^T = V^T P^T,  out = O / sum p
// with 16 tokens x 8 columns of one key/value head as one m16n8k16 product's rows and columns; a column is
// a query head of a row, and a sequence's rows x heads go in sets of 8.
// Bound by the instructions that turn the cache's codes (9/16 byte a value) into f16, a conversion and a product
// for every two values (c * s is exact in f16), twice as long as HBM needs for the bytes.  So the cache is read once
// for up to 8 columns, every lane's codes are fragments as they lie (see kv.cuh), and the
// probabilities go from the first product's result to the second's operand by a transpose of
// registers.
//
// The work is cut over the keys: all sequences' chunks of kChunk tokens, times the heads, stand in one line
// that is shared out evenly over the CTAs and inside a CTA over its warps.  A warp has its own ring of
// asynchronous copies, running maximum, sum and output, and meets the others only at its range's ends:
// parts of one (sequence, head) in one CTA are joined in shared memory, those of several CTAs in the
// workspace by the CTA that comes last, in the order of the line.  No wait for another CTA.
//
// Measured: 64 sequences of 2 to 8 thousand keys, 32 heads on 4 of 128: 50 us (3.8 TB/s), of which the
// line's set-up, the first loads and the joins are over a third; one of 131071 keys, 24 heads on 4 of 256:
// 50 us (3.0 TB/s; 8 warps a CTA, the output alone takes 64 registers a thread); 251 of up to 1500 keys,
// 64 heads on 8 of 64, window 1024: 48 us (2.6 TB/s; half the values a score has at 128).
#include <cuda_bf16.h>

#include "actq.cuh"
#include "attend.cuh"
#include "common.cuh"
#include "handle.h"
#include "kernels.h"
#include "kv.cuh"

namespace vt {

namespace {

constexpr int kHeads = 8;    // query heads of a work item: the columns of the MMA
constexpr int kStages = 2;   // chunks of a warp's ring

template <int D>
struct RowCfg {
  static constexpr int kChunk = D == 64 ? 64 : 32;          // tokens
  static constexpr int kTiles = kChunk / kKvTile;
  static constexpr int kWarps = D == 256 ? 8 : 16;
  static constexpr int kThreads = kWarps * 32;
  static constexpr int kTile = kv_tile_bytes(D);
  static constexpr int kStageBytes = kTiles * kTile;        // 4608, 4608, 9216
  static constexpr int kRing = kStages * kStageBytes;
  static constexpr int kPartFloats = kHeads * (D + 3) + 8; // O [8][D], m [8], l [8], any [8]
  static constexpr int kPartBytes = kPartFloats * 4;
  static_assert(kPartBytes <= kRing && kPartBytes % 16 == 0, "a part fits a warp's ring");
  static constexpr int kOffPart = kWarps * kRing;           // the parts that end inside a warp's range
  static constexpr int kOffMeta = kOffPart + kWarps * kPartBytes;
};

// Where a column goes in out, in elements (-1: nowhere), with its sink (-inf: none) and the global of its
// values: fetched with q, so that no join waits for them.
struct Place {
  int64_t to;
  float sink, value;
  // What the column's sums are multiplied by.
  __device__ __forceinline__ float factor(float m, float l) const { return out_factor(value, sink, m, l, kPBias); }
};
// What a warp leaves for the CTA's join: a run of chunks of one (sequence, head) line.
struct PartMeta {
  int64_t seg0;   // first chunk of the (sequence, head) on the line
  int64_t u0, u1; // chunks covered
  int nb;         // its chunks
  int used;
  const Place* place;
};
struct RowShared {
  Place place[16][2][kHeads];  // [warp][0: of its first (sequence, head, set), 1: of the one it is at]
  PartMeta part[32];       // [warp][0: ended inside the range, 1: the last]
  int64_t scan[32];
  int64_t start_prefix[16];
  int start_b[16];
  int parts, runs;         // in use, in the order of the line
  int slot[32], list[32], run_first[33];  // of each part: its place in part[], in shared memory
  float weight[32][kHeads];
  float run_m[32][kHeads], run_l[32][kHeads], run_factor[32][kHeads];
  int run_any[32][kHeads];
  int last[2];
  uint32_t lost[16 * 32];  // of each lane: columns whose sums a NaN scale reaches, 8 bits a column block
};

struct RowParams {
  AttendLaunch a;
  int G;              // CTAs
  uint32_t by_group;  // floor(2^32 / group) + 1: quotients of small numbers by it
};

// A sequence as this kernel takes it: n = 0 where the other kernel does.
struct RowSeq {
  int s0, n, len;
};
__device__ __forceinline__ RowSeq row_seq(const AttendLaunch& a, int b) {
  if (!a.starts) return {b, 1, seq_len(a, b)};
  const AttendSeq q = load_seq(a, b);
  return {q.s0, few_rows(a, q.n) ? q.n : 0, q.len};
}
// Sets of 8 columns per key/value head.
__device__ __forceinline__ int row_sets(const AttendLaunch& a, int n) { return (n * a.group + kHeads - 1) / kHeads; }
template <int D>
__device__ __forceinline__ void row_chunks(const AttendLaunch& a, const RowSeq& q, int* c0, int* nb) {
  // keys from the first that the first row sees to the last row's own
  const int64_t first = a.window > 0 ? (int64_t)q.len - q.n + 1 - a.window : 0;
  *c0 = first > 0 ? (int)(first / RowCfg<D>::kChunk) : 0;
  *nb = q.n > 0 ? (int)(((int64_t)q.len + RowCfg<D>::kChunk - 1) / RowCfg<D>::kChunk) - *c0 : 0;
}

// A chunk of the line.
template <int D>
struct Cursor {
  int b, hu, c, nb, c0, len;
  int sets, kvh;   // hu: kvh * sets + the set
  __device__ __forceinline__ int set() const { return hu - kvh * sets; }
  __device__ __forceinline__ void sequence(const RowParams& p) {
    const RowSeq q = row_seq(p.a, b);
    len = q.len;
    row_chunks<D>(p.a, q, &c0, &nb);
    sets = row_sets(p.a, q.n);
  }
  // To the next (sequence, head, set).
  __device__ __forceinline__ void next(const RowParams& p) {
    c = 0;
    kvh = ++hu / sets;
    if (kvh < p.a.cache.heads) return;
    hu = kvh = 0;
    do {
      if (++b >= p.a.B) { nb = 0; return; }
      sequence(p);
    } while (nb == 0);
  }
};

// Column i of a set (the kvh-th head's): its row of the sequence and its query head; false past the last.
// A set's columns are below 2^7: the quotient is exact.
__device__ __forceinline__ bool column_of(const RowParams& p, int n, int kvh, int set, int i, int* row, int* head) {
  const uint32_t at = set * kHeads + i;
  *row = p.a.group == 1 ? at : __umulhi(at, p.by_group);
  *head = kvh * p.a.group + at - *row * p.a.group;
  return *row < n;
}
// Keys [lo, hi) that a row of the sequence sees.
__device__ __forceinline__ int row_hi(const RowSeq& q, int row) { return max(q.len - q.n + row + 1, 0); }
__device__ __forceinline__ int row_lo(const AttendLaunch& a, int hi) {
  return a.window > 0 && a.window < hi ? hi - (int)a.window : 0;
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ uint32_t ld_shared_u32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(addr));
  return v;
}
__device__ __forceinline__ uint32_t ld_shared_u16x(uint32_t addr) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(addr));
  return v;
}

// Four A fragments' worth of codes (two words of 8) of rows g and g + 8, times their scales,
// against two k steps of Q; each has a sum of its own, so that two products run beside one another.
__device__ __forceinline__ void k_words(float (&s)[4], float (&s2)[4], uint32_t lo, uint32_t hi, uint32_t sl, uint32_t sh,
                                        const uint32_t* q) {
  uint32_t a[4], b[4];
  e2m1x8_to_f16x8(lo, a[0], a[1], a[2], a[3]);
  e2m1x8_to_f16x8(hi, b[0], b[1], b[2], b[3]);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    a[i] = hmul2_u32(a[i], sl);
    b[i] = hmul2_u32(b[i], sh);
  }
  mma_f16_16816(s, a[0], b[0], a[1], b[1], q[0], q[1]);
  mma_f16_16816(s2, a[2], b[2], a[3], b[3], q[2], q[3]);
}

// Words of codes of tokens a, b, c, d (8 columns each) and their scales, against P of a tile: four
// output tiles.
__device__ __forceinline__ void v_words(float (*o)[4], uint32_t a, uint32_t b, uint32_t c, uint32_t d,
                                        uint32_t sab, uint32_t scd, uint32_t p0, uint32_t p1) {
  constexpr uint32_t M = 0x0F0F0F0Fu;
  uint32_t e[4], f[4], g[4], h[4];
  e2m1x8_to_f16x8((a & M) | ((b << 4) & ~M), e[0], e[1], e[2], e[3]);         // even columns
  e2m1x8_to_f16x8(((a >> 4) & M) | (b & ~M), f[0], f[1], f[2], f[3]);         // odd ones
  e2m1x8_to_f16x8((c & M) | ((d << 4) & ~M), g[0], g[1], g[2], g[3]);
  e2m1x8_to_f16x8(((c >> 4) & M) | (d & ~M), h[0], h[1], h[2], h[3]);
#pragma unroll
  for (int j = 0; j < 4; ++j)
    mma_f16_16816(o[j], hmul2_u32(e[j], sab), hmul2_u32(f[j], sab), hmul2_u32(g[j], scd),
                  hmul2_u32(h[j], scd), p0, p1);
}

// Tokens of `partly` (bit 4 i + k: token t + 4 k of tile i) whose value scales, of the lane's columns,
// hold a NaN: they leave the product, where it would reach columns that do not see them, and those that do
// are noted in *lost.  Returns them, those of a second column block 16 bits up.
template <int D>
__device__ __noinline__ uint32_t nan_partly(const RowParams& p, const RowSeq& q, int kvh, int set, uint32_t st, int tok0, uint32_t partly,
                                            uint32_t* lost) {
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  uint32_t out = 0;
  for (int i = 0; i < 4 * RowCfg<D>::kTiles; ++i) {
    if (!((partly >> i) & 1)) continue;
    const int tok = tok0 + (i >> 2) * kKvTile + t + 4 * (i & 3);
    for (int c = 0; c < (D == 256 ? 2 : 1); ++c) {
      const int group = D == 64 ? g >> 1 : 8 * c + g;
      uint32_t w;
      asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w) : "r"(st + (i >> 2) * kv_tile_bytes(D) + 17 * D + group * 16 + t * 4));
      if (((w >> (8 * (i & 3))) & 0x7F) != 0x7F) continue;
      out |= 1u << (16 * c + i);
      for (int k = 0; k < kHeads; ++k) {
        int row, head;
        if (!column_of(p, q.n, kvh, set, k, &row, &head)) continue;
        const int hi = row_hi(q, row);
        if (tok >= row_lo(p.a, hi) && tok < hi) *lost |= 1u << (8 * c + k);
      }
    }
  }
  return out;
}

template <int D>
__global__ void __launch_bounds__(RowCfg<D>::kThreads, 1) k_attend_row(const RowParams p) {
  using C = RowCfg<D>;
  constexpr int NB = D == 256 ? 2 : 1;         // column blocks of a tile
  constexpr int KS = D / 16;                   // k steps of S, output tiles of O
  extern __shared__ __align__(128) uint8_t smem[];
  RowShared& sh = *reinterpret_cast<RowShared*>(smem + C::kOffMeta);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int B = (int)p.a.B;
  pdl_launch_dependents();

  // ---- the line: chunks of every sequence times its heads and sets, and where this CTA's warps begin
  auto units = [&](int b) -> int64_t {
    if (b >= B) return 0;
    const RowSeq q = row_seq(p.a, b);
    int c0, nb;
    row_chunks<D>(p.a, q, &c0, &nb);
    if (q.n > 0 && q.len == 0) {  // no key: its rows are zeros
      for (int i = blockIdx.x; i < q.n; i += gridDim.x) {
        uint4* row = reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(p.a.out) + (int64_t)(q.s0 + i) * p.a.ldo);
        for (int e = 0; e < p.a.q_heads * D / 8; ++e) row[e] = make_uint4(0, 0, 0, 0);
      }
    }
    return (int64_t)nb * (p.a.cache.heads * row_sets(p.a, q.n));
  };
  int64_t U = 0, n = 0, before = 0;
  if (B <= C::kThreads) {
    n = units(tid);
    before = block_prefix<C::kWarps>(n, sh.scan, &U);
  } else {
    for (int b = tid; b < B; b += C::kThreads) n += units(b);
    U = block_total<C::kWarps>(n, sh.scan);
  }
  if (U == 0) return;
  // a CTA has a chunk for every warp; as a multiple of the (head, set) lines, where there is room,
  // equal lines end where CTAs end (us, without and with: one sequence of 391 keys, 32 heads on 8 of 128, 14.9 and 10.2; 16 of 3000
  // 24.4 and 20.2; one of 131071, 24 on 4 of 256, 49.4 and 50.0)
  int64_t G = min((int64_t)p.G, (U + C::kWarps - 1) / C::kWarps);
  const int64_t lines = (int64_t)B * p.a.cache.heads * row_sets(p.a, 1);
  if (lines <= p.G) G = min(U, min((G + lines - 1) / lines, (int64_t)p.G / lines) * lines);
  if (blockIdx.x >= G) return;
  const int64_t cta0 = blockIdx.x * U / G, cta1 = (blockIdx.x + 1) * U / G, mine = cta1 - cta0;
  auto starts_in = [&](int b) {  // warps whose first chunk is one of sequence b's
    if (before + n <= cta0 || before >= cta1) return;
#pragma unroll 1
    for (int w = 0; w < C::kWarps; ++w) {
      const int64_t u = cta0 + mine * w / C::kWarps;
      if (u >= before && u < before + n) {
        sh.start_b[w] = b;
        sh.start_prefix[w] = before;
      }
    }
  };
  if (B <= C::kThreads) {
    starts_in(tid);
  } else {
    int64_t base = 0, round;
    for (int b0 = 0; b0 < B; b0 += C::kThreads) {
      n = units(b0 + tid);
      before = base + block_prefix<C::kWarps>(n, sh.scan, &round);
      starts_in(b0 + tid);
      base += round;
    }
  }
  if (tid < 32) sh.part[tid].used = 0;
  __syncthreads();

  const int64_t u0 = cta0 + mine * warp / C::kWarps, u1 = cta0 + mine * (warp + 1) / C::kWarps;
  const uint32_t ring = smem_u32(smem) + warp * C::kRing;
  if (u0 < u1) {
    Cursor<D> cur;
    cur.b = sh.start_b[warp];
    cur.sequence(p);
    const int64_t r = u0 - sh.start_prefix[warp];
    cur.hu = r >> 31 ? (int)(r / cur.nb) : (int)((uint32_t)r / (uint32_t)cur.nb);
    cur.kvh = cur.hu / cur.sets;
    cur.c = (int)(r - (int64_t)cur.hu * cur.nb);
    Cursor<D> ld = cur;
    const int total_chunks = (int)(u1 - u0);
    int issued = 0;
    uint32_t valid_fifo = 0;  // 4 bits per chunk in the ring: tiles that are there
    // the page of lane's tile of the chunk to be issued next, fetched ahead
    auto page_of = [&]() -> int {
      if (lane >= C::kTiles) return -1;
      const int tok = (ld.c0 + ld.c) * C::kChunk + lane * kKvTile;
      return tok < ld.len ? __ldg(p.a.tables + ld.b * p.a.ldt + (tok >> p.a.cache.page_shift)) : -1;
    };
    int page = page_of();
    auto issue = [&]() {
      const bool ok = page >= 0 && page < p.a.cache.pages;
      const int tok = (ld.c0 + ld.c) * C::kChunk + lane * kKvTile;
      const uint8_t* src = kv_tile<D>(p.a.cache, ok ? page : 0, ld.kvh, tok & (p.a.cache.page_size - 1));
      const uint32_t there = __ballot_sync(0xffffffffu, ok) & ((1u << C::kTiles) - 1);
      valid_fifo |= there << (4 * (issued < kStages ? issued : kStages - 1));
      const uint32_t dst = ring + (issued % kStages) * C::kStageBytes + lane * 16;
      constexpr int PT = C::kTile / 16;  // 16-byte pieces of a tile, 32 at a time
      const uint8_t* from[C::kTiles];
#pragma unroll
      for (int i = 0; i < C::kTiles; ++i)
        from[i] = reinterpret_cast<const uint8_t*>((uintptr_t)__shfl_sync(0xffffffffu, (uint64_t)(uintptr_t)src, i)) +
                  lane * 16 - i * C::kTile;
#pragma unroll
      for (int j = 0; j < C::kStageBytes / 512; ++j) {
        constexpr int last = C::kTiles - 1;
        const int t0 = j * 32 / PT, t1 = (j * 32 + 31) / PT < last ? (j * 32 + 31) / PT : last;
        const bool second = t1 > t0 && lane >= t1 * PT - j * 32;
        if ((there >> (second ? t1 : t0)) & 1) cp_async16(dst + j * 512, (second ? from[t1] : from[t0]) + j * 512);
      }
      ++issued;
      if (issued < total_chunks) {
        if (++ld.c == ld.nb) ld.next(p);
        page = page_of();
      }
    };

    uint32_t q[KS][2];       // B fragments: column g (a head), k = the lane's own columns
    float mul[2];            // of heads 2t and 2t + 1: raw products to log2 units
    float o[KS][4], m[2], l[2];
    uint32_t any = 0;         // bit i: column 2t + i has seen a key
    int first_c = cur.c, all_lo, all_hi;   // keys [all_lo, all_hi) are seen by every column
    int later = 0;            // past the warp's first (sequence, head, set)
    auto load_q = [&](uint4 (&w)[KS / 2]) {
      const RowSeq sq = row_seq(p.a, cur.b);
      int row, head;
      const bool on = column_of(p, sq.n, cur.kvh, cur.set(), g, &row, &head);
      if (t == 0) {
        Place& to = sh.place[warp][later][g];
        to.to = on ? (int64_t)(sq.s0 + row) * p.a.ldo + (int64_t)head * D : -1;
        to.sink = on && p.a.sinks ? __ldg(p.a.sinks + head) : -INFINITY;
        to.value = __ldg(p.a.cache.v_scale + cur.kvh);
      }
      const __nv_bfloat16* src = reinterpret_cast<const __nv_bfloat16*>(p.a.q) + (on ? (int64_t)(sq.s0 + row) * p.a.ldq + (int64_t)head * D : 0) +
                                 (D == 64 ? 16 : 32) * t;
#pragma unroll
      for (int i = 0; i < KS / 2; ++i) {
        w[i] = make_uint4(0, 0, 0, 0);
        if (on) w[i] = *reinterpret_cast<const uint4*>(src + (D == 256 ? (i >> 2) * 128 + (i & 3) * 8 : i * 8));
      }
    };
    auto begin = [&](uint4 (&w)[KS / 2]) {
      const RowSeq sq = row_seq(p.a, cur.b);
      int mx = 0;
#pragma unroll
      for (int i = 0; i < KS / 2; ++i) mx = max(mx, act_maxmag8(reinterpret_cast<const uint32_t*>(&w[i])));
      mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      const int pw = act_pow2(mx);
#pragma unroll
      for (int i = 0; i < KS / 2; ++i) {
        const uint4 f = act_granule_f16(reinterpret_cast<const uint32_t*>(&w[i]), pw);
        q[2 * i][0] = f.x, q[2 * i][1] = f.y, q[2 * i + 1][0] = f.z, q[2 * i + 1][1] = f.w;
      }
      int h0, r0, r1;
      column_of(p, sq.n, cur.kvh, cur.set(), 0, &r0, &h0);
      const float unit = p.a.scale * kLog2e * __ldg(p.a.cache.k_scale + cur.kvh);
      // the set's first and last row bound what all of them see
      column_of(p, sq.n, cur.kvh, cur.set(), kHeads - 1, &r1, &h0);
      r1 = min(r1, sq.n - 1);
      all_hi = row_hi(sq, r0);
      all_lo = row_lo(p.a, row_hi(sq, r1));
      sh.lost[tid] = 0;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        mul[i] = unit * pow2f(__shfl_sync(0xffffffffu, pw, 4 * (2 * t + i)));
        m[i] = -INFINITY;
        l[i] = 0.0f;
      }
#pragma unroll
      for (int j = 0; j < KS; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[j][e] = 0.0f;
      any = 0;
      first_c = cur.c;
    };
    // loads of q and of the first page's entry are in flight together
    uint4 w0[KS / 2];
    load_q(w0);
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) {
      if (issued < total_chunks) issue();
      cp_commit();
    }
    begin(w0);

#pragma unroll 1
    for (int n = 0; n < total_chunks; ++n) {
      if (issued < total_chunks) issue();
      cp_commit();
      cp_wait<kStages - 1>();
      __syncwarp();
      const uint32_t st = ring + (n % kStages) * C::kStageBytes;
      const uint32_t there = valid_fifo & 15u;
      valid_fifo >>= 4;
      const int tok0 = (cur.c0 + cur.c) * C::kChunk;
      const bool edge = tok0 < all_lo || tok0 + C::kChunk > all_hi || there != (1u << C::kTiles) - 1;

      // ---- S^T = K Q^T
      float s[C::kTiles][4];
#pragma unroll
      for (int i = 0; i < C::kTiles; ++i) {
        const uint32_t tb = st + i * C::kTile;
#pragma unroll
        for (int e = 0; e < 4; ++e) s[i][e] = 0.0f;
        float s2[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        if constexpr (D == 64) {
          const uint2 lo = ld_shared_v2(tb + g * 32 + t * 8), hi = ld_shared_v2(tb + 256 + g * 32 + t * 8);
          const uint32_t sc = e4m3x2_to_f16x2(ld_shared_u16x(tb + 8 * D + g * 8 + t * 2));
          const uint32_t sl = bcast_lo(sc), sr = bcast_hi(sc);
          k_words(s[i], s2, lo.x, hi.x, sl, sr, q[0]);
          k_words(s[i], s2, lo.y, hi.y, sl, sr, q[2]);
        } else {
#pragma unroll
          for (int c = 0; c < NB; ++c) {
            const int4 lo = ld_shared_v4(tb + c * 1024 + g * 64 + t * 16);
            const int4 hi = ld_shared_v4(tb + c * 1024 + 512 + g * 64 + t * 16);
            const uint32_t sw = ld_shared_u32(tb + 8 * D + c * 128 + g * 16 + t * 4);
            const uint32_t s0 = e4m3x2_to_f16x2(sw), s1 = e4m3x2_to_f16x2(sw >> 16);
            k_words(s[i], s2, lo.x, hi.x, bcast_lo(s0), bcast_lo(s1), q[8 * c]);
            k_words(s[i], s2, lo.y, hi.y, bcast_lo(s0), bcast_lo(s1), q[8 * c + 2]);
            k_words(s[i], s2, lo.z, hi.z, bcast_hi(s0), bcast_hi(s1), q[8 * c + 4]);
            k_words(s[i], s2, lo.w, hi.w, bcast_hi(s0), bcast_hi(s1), q[8 * c + 6]);
          }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) s[i][e] = (s[i][e] + s2[e]) * mul[e & 1];
      }
      // ---- keys that a column does not see; what their places hold may be anything
      uint32_t seen = 0xFFFFFFFFu;  // bit 16 c + 4 i + k: token t + 4 k of tile i, column block c, by some column
      if (edge) {
        const RowSeq sq = row_seq(p.a, cur.b);
        int row, head, lo[2], hi[2];
        column_of(p, sq.n, cur.kvh, cur.set(), 2 * t, &row, &head);
        hi[0] = row < sq.n ? row_hi(sq, row) : 0;
        lo[0] = row_lo(p.a, hi[0]);
        column_of(p, sq.n, cur.kvh, cur.set(), 2 * t + 1, &row, &head);
        hi[1] = row < sq.n ? row_hi(sq, row) : 0;
        lo[1] = row_lo(p.a, hi[1]);
        bool some[2] = {false, false};
#pragma unroll
        for (int i = 0; i < C::kTiles; ++i) {
          const int a = tok0 + i * kKvTile + kv_mma_token(g), b = tok0 + i * kKvTile + kv_mma_token(g + 8);
          const bool in = (there >> i) & 1;
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const bool sa = in && a >= lo[k] && a < hi[k], sb = in && b >= lo[k] && b < hi[k];
            some[k] |= sa || sb;
            s[i][k] = sa ? s[i][k] : -INFINITY;
            s[i][2 + k] = sb ? s[i][2 + k] : -INFINITY;
          }
        }
        seen = 0;
        const int last = row_hi(sq, sq.n - 1), first = row_lo(p.a, row_hi(sq, 0));
        uint32_t partly = 0;           // of those, not by all of the set
#pragma unroll
        for (int i = 0; i < C::kTiles; ++i)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int tok = tok0 + i * kKvTile + t + 4 * k;
            if (((there >> i) & 1) && tok >= first && tok < last) {
              seen |= 1u << (4 * i + k);
              if (tok < all_lo || tok >= all_hi) partly |= 1u << (4 * i + k);
            }
          }
        // a column has seen a key: bits 2 t, 2 t + 1 of its lanes, for all of them
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const uint32_t who = __ballot_sync(0xffffffffu, some[k]);
          if (who & (0x11111111u << t)) any |= 1u << k;
        }
        if (NB == 2) seen |= seen << 16;
        if (__any_sync(0xffffffffu, partly != 0)) seen &= ~nan_partly<D>(p, sq, cur.kvh, cur.set(), st, tok0, partly, &sh.lost[tid]);
      } else {
        any = 3;
      }
      // ---- running maximum: the sums stay on an older one while no lane has a score more than kSlack
      // above it, so that the maximum over the lanes and the scaling are rare
      float top[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        top[i] = fmaxf(s[0][i], s[0][i + 2]);
#pragma unroll
        for (int j = 1; j < C::kTiles; ++j) top[i] = fmaxf(top[i], fmaxf(s[j][i], s[j][i + 2]));
      }
      if (__any_sync(0xffffffffu, top[0] > m[0] + kSlack || top[1] > m[1] + kSlack)) {
        float f[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float x = top[i];
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
          f[i] = x > m[i] ? fast_exp2(m[i] - x) : 1.0f;
          l[i] *= f[i];
          m[i] = fmaxf(m[i], x);
        }
#pragma unroll
        for (int j = 0; j < KS; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[j][e] *= f[e & 1];
      }
      const float off[2] = {kPBias - (m[0] == -INFINITY ? 0.0f : m[0]), kPBias - (m[1] == -INFINITY ? 0.0f : m[1])};
      // ---- O^T += V^T P^T
#pragma unroll
      for (int i = 0; i < C::kTiles; ++i) {
        float pr[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          pr[e] = fast_exp2(s[i][e] + off[e & 1]);
          l[e & 1] += pr[e];
        }
        const uint32_t p0 = transpose8x8(pack_half2(pr[0], pr[1])), p1 = transpose8x8(pack_half2(pr[2], pr[3]));
        const uint32_t tb = st + i * C::kTile + 9 * D;
        auto scales = [&](int group, int c) {
          uint32_t w = ld_shared_u32(tb + 8 * D + group * 16 + t * 4);
          if (edge) {  // a place that is not seen may hold a NaN scale
            const uint32_t k = seen >> (16 * c + 4 * i);
            w &= ((k & 1) ? 0xFFu : 0u) | ((k & 2) ? 0xFF00u : 0u) | ((k & 4) ? 0xFF0000u : 0u) | ((k & 8) ? 0xFF000000u : 0u);
          }
          return w;
        };
        if constexpr (D == 64) {
          const uint32_t at = tb + t * 32 + g * 4;
          const uint32_t sw = scales(g >> 1, 0);
          v_words(o, ld_shared_u32(at), ld_shared_u32(at + 128), ld_shared_u32(at + 256), ld_shared_u32(at + 384),
                  e4m3x2_to_f16x2(sw), e4m3x2_to_f16x2(sw >> 16), p0, p1);
        } else {
#pragma unroll
          for (int c = 0; c < NB; ++c) {
            const uint32_t at = tb + c * 1024 + t * 64 + ((g * 8) ^ ((t >> 1) * 32));
            const uint2 a = ld_shared_v2(at), b = ld_shared_v2(at + 256), cc = ld_shared_v2(at + 512), d = ld_shared_v2(at + 768);
            const uint32_t sw = scales(8 * c + g, c);
            const uint32_t sab = e4m3x2_to_f16x2(sw), scd = e4m3x2_to_f16x2(sw >> 16);
            v_words(o + 8 * c, a.x, b.x, cc.x, d.x, sab, scd, p0, p1);
            v_words(o + 8 * c + 4, a.y, b.y, cc.y, d.y, sab, scd, p0, p1);
          }
        }
      }
      __syncwarp();  // every lane has read the stage before it is filled again

      // ---- the end of this (sequence, head), or of the warp's range
      const bool ends = cur.c + 1 == cur.nb, last = n + 1 == total_chunks;
      if (ends || last) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          l[i] += __shfl_xor_sync(0xffffffffu, l[i], 4);
          l[i] += __shfl_xor_sync(0xffffffffu, l[i], 8);
          l[i] += __shfl_xor_sync(0xffffffffu, l[i], 16);
        }
        constexpr int EJ = D == 64 ? 4 : 8;   // output tiles of a column block
        uint32_t lost = sh.lost[tid];         // met by the lanes of this column group
        lost |= __shfl_xor_sync(0xffffffffu, lost, 1);
        lost |= __shfl_xor_sync(0xffffffffu, lost, 2);
        if (lost) {
#pragma unroll
          for (int j = 0; j < KS; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if ((lost >> (8 * (j >> 3) + 2 * t + (e & 1))) & 1) o[j][e] = __uint_as_float(0x7FC00000u);
        }
        if (ends && first_c == 0) {           // all of it
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const bool some = (any >> i) & 1;
            const Place at = sh.place[warp][later][2 * t + i];
            const float f = at.factor(m[i], l[i]);
            if (at.to >= 0) {
              __nv_bfloat16* dst = reinterpret_cast<__nv_bfloat16*>(p.a.out) + at.to;
#pragma unroll
              for (int c = 0; c < NB; ++c) {
                uint32_t w[EJ];
#pragma unroll
                for (int j = 0; j < EJ; ++j) {
                  const float x = some ? o[8 * c + j][i] * f : 0.0f, y = some ? o[8 * c + j][i + 2] * f : 0.0f;
                  const __nv_bfloat162 v = __floats2bfloat162_rn(x, y);
                  w[j] = *reinterpret_cast<const uint32_t*>(&v);
                }
#pragma unroll
                for (int j = 0; j < EJ; j += 4)
                  *reinterpret_cast<uint4*>(dst + c * 128 + (2 * EJ) * g + 2 * j) = make_uint4(w[j], w[j + 1], w[j + 2], w[j + 3]);
              }
            }
          }
        } else {
          // ends inside the range (it began before it): a place of its own; else the warp's ring,
          // which no copy is under way to any more
          const int kind = ends && !last ? 0 : 1;
          float* part = reinterpret_cast<float*>(smem + (kind ? warp * C::kRing : C::kOffPart + warp * C::kPartBytes));
          cp_wait_all_if(kind);
#pragma unroll
          for (int c = 0; c < NB; ++c)
#pragma unroll
            for (int j = 0; j < EJ; ++j)
#pragma unroll
              for (int i = 0; i < 2; ++i)
                *reinterpret_cast<float2*>(part + (2 * t + i) * D + c * 128 + 2 * EJ * g + 2 * j) =
                    make_float2(o[8 * c + j][i], o[8 * c + j][i + 2]);
          if (g == 0) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              part[kHeads * D + 2 * t + i] = m[i];
              part[kHeads * D + kHeads + 2 * t + i] = l[i];
            }
          }
          if (g == 0) {
            part[kHeads * D + 2 * kHeads + 2 * t] = any & 1 ? 1.0f : 0.0f;
            part[kHeads * D + 2 * kHeads + 2 * t + 1] = any & 2 ? 1.0f : 0.0f;
          }
          if (lane == 0) {
            PartMeta& pm = sh.part[2 * warp + kind];
            pm.seg0 = u0 + n - cur.c;
            pm.u0 = u0 + n - cur.c + first_c;
            pm.u1 = u0 + n + 1;
            pm.nb = cur.nb;
            pm.place = sh.place[warp][later];
            pm.used = 1;
          }
        }
        if (!last) {
          cur.next(p);
          later = 1;
          __syncwarp();  // every lane has read the places that are filled again
          uint4 w[KS / 2];
          load_q(w);
          begin(w);
        }
      } else {
        ++cur.c;
      }
    }
  }
  __syncthreads();

  // ---- join the parts of each (sequence, head, set): runs of neighbours in the order of the line
  if (warp == 0) {
    const bool used = lane < 2 * C::kWarps && sh.part[lane].used;
    const uint32_t all = __ballot_sync(0xffffffffu, used), below = all & ((1u << lane) - 1);
    const bool first = used && (!below || sh.part[31 - __clz(below)].seg0 != sh.part[lane].seg0);
    const uint32_t firsts = __ballot_sync(0xffffffffu, first);
    const int k = __popc(below), run = __popc(firsts & ((2u << lane) - 1)) - 1;
    if (used) {
      sh.slot[k] = lane;
      sh.list[k] = (lane & 1) ? (lane >> 1) * C::kRing : C::kOffPart + (lane >> 1) * C::kPartBytes;
    }
    if (first) sh.run_first[run] = k;
    if (lane == 0) {
      sh.parts = __popc(all);
      sh.runs = __popc(firsts);
      sh.run_first[__popc(firsts)] = __popc(all);
    }
  }
  __syncthreads();
  const int runs = sh.runs;
  auto part_at = [&](int k) { return reinterpret_cast<const float*>(smem + sh.list[k]); };
  // a warp takes one column of a run: its parts side by side in the lanes
#pragma unroll 1
  for (int task = warp; task < runs * kHeads; task += C::kWarps) {
    const int run = task / kHeads, h = task % kHeads, k0 = sh.run_first[run], n = sh.run_first[run + 1] - k0;
    const Place& at = sh.part[sh.slot[k0]].place[h];
    const float* q = part_at(k0 + (lane < n ? lane : 0)) + kHeads * D + h;
    const float mine = q[0];
    float m = mine;
#pragma unroll
    for (int k = 16; k; k >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, k));
    const float w = fast_exp2(mine - (m == -INFINITY ? 0.0f : m));
    float l = lane < n ? w * q[kHeads] : 0.0f;
#pragma unroll
    for (int k = 16; k; k >>= 1) l += __shfl_xor_sync(0xffffffffu, l, k);
    const bool any = __any_sync(0xffffffffu, q[2 * kHeads] != 0.0f);
    if (lane < n) sh.weight[k0 + lane][h] = w;
    if (lane == 0) {
      sh.run_m[run][h] = m;
      sh.run_l[run][h] = l;
      sh.run_any[run][h] = any;
      sh.run_factor[run][h] = at.factor(m, l);
    }
  }
  __syncthreads();
  auto store_pair = [&](const PartMeta& first, int at, float2 o, const float* factor, const int* some) {
    const int h = at / D;
    const int64_t to = first.place[h].to;
    const float f = factor[h];
    const bool any = some[h];
    if (to >= 0)
      *reinterpret_cast<__nv_bfloat162*>(reinterpret_cast<__nv_bfloat16*>(p.a.out) + to + at % D) =
          any ? __floats2bfloat162_rn(o.x * f, o.y * f) : __floats2bfloat162_rn(0.0f, 0.0f);
  };
  float* parts = reinterpret_cast<float*>(p.a.workspace + kAttendCleared);
  uint32_t* counters = reinterpret_cast<uint32_t*>(p.a.workspace + kRowCounts);
  constexpr int kPairs = kHeads * D / 2;  // of a run's sums
  auto whole = [&](int run) {
    const PartMeta &f = sh.part[sh.slot[sh.run_first[run]]], &e = sh.part[sh.slot[sh.run_first[run + 1] - 1]];
    return f.u0 == f.seg0 && e.u1 == f.seg0 + f.nb;
  };
#pragma unroll 1
  for (int i = tid; i < runs * kPairs; i += C::kThreads) {
    const int run = i / kPairs, at = (i % kPairs) * 2, h = at / D;
    float2 o = make_float2(0.0f, 0.0f);
#pragma unroll 4
    for (int k = sh.run_first[run]; k < sh.run_first[run + 1]; ++k) {
      const float w = sh.weight[k][h];
      const float2 v = *reinterpret_cast<const float2*>(part_at(k) + at);
      o.x += w * v.x;
      o.y += w * v.y;
    }
    const PartMeta& first = sh.part[sh.slot[sh.run_first[run]]];
    if (whole(run)) {
      store_pair(first, at, o, sh.run_factor[run], sh.run_any[run]);
    } else {
      // slot 0: what began in an earlier CTA, slot 1: what begins here and goes on
      float* dst = parts + ((int64_t)blockIdx.x * 2 + (first.u0 == first.seg0)) * C::kPartFloats;
      __stcg(reinterpret_cast<float2*>(dst + at), o);
      if (at % D == 0) {
        __stcg(dst + kHeads * D + h, sh.run_m[run][h]);
        __stcg(dst + kHeads * D + kHeads + h, sh.run_l[run][h]);
        __stcg(dst + kHeads * D + 2 * kHeads + h, sh.run_any[run][h] ? 1.0f : 0.0f);
      }
    }
  }
  // ---- parts that other CTAs hold too (of the first run, of the last): the last one to come joins them
  const bool shared0 = runs > 0 && !whole(0), shared1 = runs > 1 && !whole(runs - 1);
  if (!shared0 && !shared1) return;
  // CTAs from c0 to c1 share a run: CTA i holds [i U / G, (i + 1) U / G)
  auto first_cta = [&](const PartMeta& f) { return ((f.seg0 + 1) * G - 1) / U; };
  auto last_cta = [&](const PartMeta& f) { return ((f.seg0 + f.nb) * G - 1) / U; };
  __syncthreads();  // the fence below covers what the CTA wrote before
  if (lane == 0 && warp < 2) {
    sh.last[warp] = 0;
    if (warp ? shared1 : shared0) {
      const PartMeta& f = sh.part[sh.slot[sh.run_first[warp ? runs - 1 : 0]]];
      uint32_t* count = counters + first_cta(f);
      __threadfence();
      const bool last = atomicAdd(count, 1u) == (uint32_t)(last_cta(f) - first_cta(f));
      if (last) *count = 0;  // for the next call
      __threadfence();
      sh.last[warp] = last;
    }
  }
  __syncthreads();
  float* weight = reinterpret_cast<float*>(smem);  // [parts][8], in the place of the rings
#pragma unroll 1
  for (int which = 0; which < 2; ++which) {
    if (!sh.last[which]) continue;
    const PartMeta& f = sh.part[sh.slot[sh.run_first[which ? runs - 1 : 0]]];
    const int64_t c0 = first_cta(f);
    const int n = (int)(last_cta(f) - c0) + 1;
    // CTA c0's part is in its slot 1, the others' in their slot 0
    auto part_of = [&](int k) { return parts + (2 * (c0 + k) + (k == 0)) * (int64_t)C::kPartFloats; };
    for (int h = warp; h < kHeads; h += C::kWarps) {
      float m = -INFINITY, l = 0.0f;
      bool any = false;
#pragma unroll 1
      for (int k = lane; k < n; k += 32) m = fmaxf(m, __ldcg(part_of(k) + kHeads * D + h));
#pragma unroll
      for (int k = 16; k; k >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, k));
      const float ms = m == -INFINITY ? 0.0f : m;
#pragma unroll 1
      for (int k = lane; k < n; k += 32) {
        const float* q = part_of(k) + kHeads * D + h;
        const float w = fast_exp2(__ldcg(q) - ms);
        weight[k * kHeads + h] = w;
        l += w * __ldcg(q + kHeads);
        any |= __ldcg(q + 2 * kHeads) != 0.0f;
      }
#pragma unroll
      for (int k = 16; k; k >>= 1) l += __shfl_xor_sync(0xffffffffu, l, k);
      any = __any_sync(0xffffffffu, any);
      if (lane == 0) {
        sh.run_any[which][h] = any;
        sh.run_factor[which][h] = f.place[h].factor(m, l);
      }
    }
    __syncthreads();
    for (int i = tid; i < kPairs; i += C::kThreads) {
      const int at = i * 2, h = at / D;
      float2 o = make_float2(0.0f, 0.0f);
#pragma unroll 4
      for (int k = 0; k < n; ++k) {
        const float2 v = __ldcg(reinterpret_cast<const float2*>(part_of(k) + at));
        const float w = weight[k * kHeads + h];
        o.x += w * v.x;
        o.y += w * v.y;
      }
      store_pair(f, at, o, sh.run_factor[which], sh.run_any[which]);
    }
    __syncthreads();
  }
}

template <int D>
cudaError_t go(const RowParams& p, cudaStream_t s) {
  using C = RowCfg<D>;
  static int done[64];
  constexpr size_t bytes = C::kOffMeta + sizeof(RowShared);
  static_assert(bytes <= 232448, "shared memory");
  if (cudaError_t e = set_up_kernel(k_attend_row<D>, bytes, done)) return e;
  k_attend_row<D><<<p.G, C::kThreads, bytes, s>>>(p);
  return cudaGetLastError();
}

}  // namespace

size_t attend_row_parts_bytes(int head_dim) {
  const size_t f = head_dim == 64 ? RowCfg<64>::kPartBytes : head_dim == 128 ? RowCfg<128>::kPartBytes : RowCfg<256>::kPartBytes;
  return 2 * (size_t)kMaxAttendGrid * f;
}

cudaError_t launch_attend_row(const AttendLaunch& L, int head_dim, cudaStream_t s) {
  RowParams p;
  p.a = L;
  p.G = sm_count() < kMaxAttendGrid ? sm_count() : kMaxAttendGrid;
  p.by_group = (uint32_t)(((uint64_t)1 << 32) / L.group + 1);
  return head_dim == 64 ? go<64>(p, s) : head_dim == 128 ? go<128>(p, s) : go<256>(p, s);
}

}  // namespace vt
