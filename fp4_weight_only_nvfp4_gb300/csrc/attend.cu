// Which kernel serves a call of attention over the paged NVFP4 cache.
#include "attend.cuh"

namespace vt {

// Calls of up to T rows: with so few none of their sequences is the tile kernel's.
static bool tiles(int64_t T, int group) { return T * group > kFewColumns; }

// Each kernel has its parts and its arrival counts.
size_t attend_workspace_bytes(int64_t T, int group, int head_dim) {
  return kAttendCleared + attend_row_parts_bytes(head_dim) + (tiles(T, group) ? attend_tile_parts_bytes(head_dim) : 0);
}

cudaError_t launch_attend(const AttendLaunch& L, int head_dim, cudaStream_t s) {
  if (cudaError_t e = launch_attend_row(L, head_dim, s)) return e;
  // no sequence has more rows than the call (4 rows of 32 heads on 8 of 128 behind 2000 keys: 14.4 us, 16.6 with
  // both kernels)
  return L.starts && tiles(L.T, L.group) ? launch_attend_tile(L, head_dim, s) : cudaSuccess;
}

}  // namespace vt
