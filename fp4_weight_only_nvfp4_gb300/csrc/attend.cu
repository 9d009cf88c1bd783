// Which kernel serves a call of attention over the paged NVFP4 cache.
#include "attend.cuh"

namespace vt {

size_t attend_workspace_bytes(int64_t T, int64_t B, int q_heads, int heads, int head_dim) {
  const size_t row = attend_row_parts_bytes(head_dim), tile = attend_tile_parts_bytes(head_dim);
  return kAttendCleared + (row > tile ? row : tile);
}

cudaError_t launch_attend(const AttendLaunch& L, int head_dim, cudaStream_t s) {
  return L.starts ? launch_attend_tile(L, head_dim, s) : launch_attend_row(L, head_dim, s);
}

}  // namespace vt
