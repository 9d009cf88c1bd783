// The paged NVFP4 cache of keys and values: where each code and scale byte stands.
//
// A page holds, for each key/value head, its tokens in tiles of 16; a tile is one run of bytes, so that
// a copy of n tiles of a page is one copy.  For head_dim D a tile is 18 * D bytes:
//   K codes at 0, K scales at 8 D, V codes at 9 D, V scales at 17 D.
// D = 256 is two column blocks of 128 beside one another in each of the four parts (W = min(D,
// 128) columns a block).  Inside a block the bytes stand in the order of the fragments of the
// decode kernel's m16n8k16 products, K as the A operand of S^T = K Q^T and V^T as that of O^T =
// V^T P^T, lane l = 4 g + t:
//   K rows are stored in the order of the MMA's rows: token r at row kv_mma_row(r), W / 2 bytes each.  Lane (g, t) reads the t-th
//     quarter of rows g and g + 8 (W / 8 bytes, 16 at D >= 128: one load each).
//   K scales: a word for each (g, t) at D >= 128 holds the two scales of the quarter for row g and for
//     row g + 8 (D = 64: 16 bits, one scale each).
//   V rows are in token order, W / 2 bytes each; lane (g, t) reads the g-th eighth of tokens t, 4 + t, 8
//     + t and 12 + t.  At W = 128 the two 32-byte halves of a row change places where bit 1 of the
//     token is set, so that the 16 lanes of a half warp meet no bank twice.
//   V scales: the word (scale group, t) holds those of tokens t, 4 + t, 8 + t, 12 + t.
// The order of tokens among the MMA's rows and k columns is free as long as both products use the
// same one: with token t + 4 i at row {2t, 2t + 1, 2t + 8, 2t + 9}[i] the four tokens whose
// probabilities a lane holds as its B fragment are the four whose scales are one word.
#pragma once
#include <stdint.h>

namespace vt {

constexpr int kKvTile = 16;  // tokens

__host__ __device__ constexpr int kv_tile_bytes(int D) { return 18 * D; }

// Row of the MMA that token r of a tile takes, and the token at a row.
__host__ __device__ constexpr int kv_mma_row(int r) { return 2 * (r & 3) + ((r >> 2) & 1) + 8 * (r >> 3); }
__host__ __device__ constexpr int kv_mma_token(int row) {
  return ((row & 7) >> 1) + 4 * (row & 1) + 8 * (row >> 3);
}

// Byte of a tile holding codes 2 b and 2 b + 1 of token r (b < D / 2), and scale s (s < D / 16).
__host__ __device__ constexpr int kv_k_code(int D, int r, int b) {
  return D == 64 ? kv_mma_row(r) * 32 + b : (b >> 6) * 1024 + kv_mma_row(r) * 64 + (b & 63);
}
__host__ __device__ constexpr int kv_k_scale(int D, int r, int s) {
  return 8 * D + (D == 64 ? (kv_mma_row(r) & 7) * 8 + s * 2 + (kv_mma_row(r) >> 3)
                          : (s >> 3) * 128 + (kv_mma_row(r) & 7) * 16 + ((s & 7) >> 1) * 4 +
                                (kv_mma_row(r) >> 3) * 2 + (s & 1));
}
__host__ __device__ constexpr int kv_v_code(int D, int r, int b) {
  return 9 * D + (D == 64 ? r * 32 + b
                          : (b >> 6) * 1024 + r * 64 + ((b & 63) ^ (((r >> 1) & 1) * 32)));
}
__host__ __device__ constexpr int kv_v_scale(int D, int r, int s) {
  return 17 * D + s * 16 + (r & 3) * 4 + (r >> 2);
}

// The cache as the kernels see it.
struct KvCache {
  uint8_t* data;
  int64_t page_stride;
  int64_t slots;      // pages * page_size
  int pages, heads;
  int page_size, page_shift;
  const float* k_scale;
  const float* v_scale;
};

// Tile holding token `in` of page `page`, for head h.
template <int D>
__device__ __forceinline__ uint8_t* kv_tile(const KvCache& c, int64_t page, int h, int in) {
  return c.data + page * c.page_stride +
         ((int64_t)h * (c.page_size / kKvTile) + in / kKvTile) * kv_tile_bytes(D);
}

}  // namespace vt
