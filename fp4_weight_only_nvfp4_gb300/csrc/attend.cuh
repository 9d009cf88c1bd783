// Shared by the kernels of attention over the paged NVFP4 cache.
#pragma once
#include "kernels.h"

namespace vt {

constexpr int kAttendCleared = 4096;  // status word and arrival counts, zeros between calls
constexpr int kMaxAttendGrid = 160;
constexpr int kRowCounts = 256, kTileCounts = 2048;  // of the arrival counts, bytes
static_assert(kRowCounts + 4 * kMaxAttendGrid <= kTileCounts && kTileCounts + 4 * kMaxAttendGrid <= kAttendCleared, "counts");
constexpr float kLog2e = 1.4426950408889634f;
// Probabilities are held as 2^(s - m + kPBias) with m the row's maximum or an older one that it passes
// by kSlack at most: below 2^15 in f16, and those down to 2^-21 of the largest keep all their
// bits (2^-31: the last bit), so that a long row's sum keeps what many small ones add.
// They are rounded to f16 for the second product, whose operands have 16 bits; scores, the softmax's sums and the output stay
// in fp32.  The rounding (2^-11 of each, of either sign) moves an output by some hundredth of the step of its one
// rounding to bf16: some 2 % of them take the neighbour, and the error against 64 bits stays that of the rounding to bf16
// alone, 0.0016 to 0.0017 of the outputs' norm.  Two f16 a probability would double the second product.
constexpr float kPBias = 7.0f, kSlack = 8.0f;

__device__ __forceinline__ float fast_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void cp_wait_all_if(bool yes) {
  if (yes) asm volatile("cp.async.wait_all;" ::: "memory");
}

// Keys of sequence b.
__device__ __forceinline__ int seq_len(const AttendLaunch& a, int64_t b) {
  const int64_t most = a.ldt << a.cache.page_shift, n = __ldg(a.lens + b);
  return (int)(n < 0 ? 0 : n > most ? most : n);
}
// Its rows and keys, whatever starts and lens hold.
struct AttendSeq {
  int s0, n, len;
};
__device__ __forceinline__ AttendSeq load_seq(const AttendLaunch& a, int64_t b) {
  AttendSeq q;
  const int T = (int)a.T, s = __ldg(a.starts + b), e = __ldg(a.starts + b + 1);
  q.s0 = s < 0 ? 0 : s > T ? T : s;
  q.n = (e < q.s0 ? q.s0 : e > T ? T : e) - q.s0;
  q.len = seq_len(a, b);
  return q;
}
// Which kernel takes a sequence of n rows (with starts): up to kFewColumns rows x query heads of a
// key/value head go 8 at a time through the row kernel, more as tiles of 128 rows.  us, as columns and as tiles, 31 sequences
// behind 3000 keys: 32 heads on 4 of 128, 16 rows x heads 34 and 62, 32 57 and 61, 40 68 and 61, 64 101 and 61; 32 on 8 of
// 128, 32 92 and 114, 40 113 and 116, 48 131 and 116; 64 on 8 of 64, 32 58 and 75, 40 69 and 76, 48 79 and 77; 24 on 4 of 256, 24 80 and 98,
// 48 151 and 101.  (A single sequence would be faster as columns up to 64: 22 and 46 behind 3000 keys, 32 on 8 of 128.)
constexpr int kFewColumns = 32;
__device__ __forceinline__ bool few_rows(const AttendLaunch& a, int n) { return (int64_t)n * a.group <= kFewColumns; }

// What a row's sum of p v is multiplied by: the values' global over the sum of p and the sink's
// share (m in log2 units; p and l hold 2^bias; a sink of -inf is none).
__device__ __forceinline__ float out_factor(float value, float sink, float m, float l, float bias) {
  const float s = sink * kLog2e, top = fmaxf(m, s), ts = top == -INFINITY ? 0.0f : top;
  const float w = fast_exp2(m - ts);  // the row's sums are re-based where the sink is larger
  return value * w / (l * w + fast_exp2(s - ts + bias));
}
// Sum over the CTA's threads, and the sum over the threads before this one.
template <int WARPS>
__device__ __forceinline__ int64_t block_prefix(int64_t v, int64_t* scan, int64_t* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t x = v;
#pragma unroll
  for (int k = 1; k < 32; k <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, x, k);
    if (lane >= k) x += y;
  }
  __syncthreads();
  if (lane == 31) scan[warp] = x;
  __syncthreads();
  int64_t before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < WARPS; ++w) {
    if (w < warp) before += scan[w];
    all += scan[w];
  }
  *total = all;
  return before + x - v;
}
template <int WARPS>
__device__ __forceinline__ int64_t block_total(int64_t v, int64_t* scan) {
  int64_t all;
  block_prefix<WARPS>(v, scan, &all);
  return all;
}

// Bytes of the parts that CTAs hand to one another.
size_t attend_row_parts_bytes(int head_dim);
size_t attend_tile_parts_bytes(int head_dim);
cudaError_t launch_attend_row(const AttendLaunch& L, int head_dim, cudaStream_t s);
cudaError_t launch_attend_tile(const AttendLaunch& L, int head_dim, cudaStream_t s);

}  // namespace vt
