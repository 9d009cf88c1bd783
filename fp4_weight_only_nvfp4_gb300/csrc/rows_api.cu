// C entry points of the operators on rows grouped by an index (declared in include/vt_fp4.h):
// the router, the grouping, the ragged products and the low-rank adapters.  Argument checks
// run before any CUDA call.
#include <limits.h>
#include <math.h>
#include <stdarg.h>
#include <stdio.h>

#include "common.cuh"
#include "handle.h"
#include "kernels.h"
#include "vt_fp4.h"

using namespace vt;

namespace {

vt_status fail(vt_status st, const char* fmt, ...) {
  char msg[256];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(msg, sizeof(msg), fmt, ap);
  va_end(ap);
  return set_last_error(st, msg);
}

vt_status done(cudaError_t e, const char* where) {
  if (e == cudaSuccess) return VT_OK;
  return fail(VT_ERR_CUDA, "%s: %s (%s)", where, cudaGetErrorName(e), cudaGetErrorString(e));
}

inline bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }
inline size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }
// A group of n rows is cut into nt tiles of 16 rows or more, and the kernels' n + nt + 128 stays an int.
constexpr int64_t kMaxPairs = ((int64_t)1 << 31) - ((int64_t)1 << 27);

vt_status check_groups(int64_t pairs, int64_t E) {
  if (E < 1 || E > kMaxGroups) return fail(VT_ERR_INVALID_ARG, "E must be in [1, %d]", kMaxGroups);
  if (pairs < 0 || pairs >= kMaxPairs)
    return fail(VT_ERR_INVALID_ARG, "pairs must be in [0, 2^31 - 2^27) (got %lld)", (long long)pairs);
  return VT_OK;
}

vt_status check_workspace(const void* ws, size_t have, size_t need) {
  if (!ws) return fail(VT_ERR_INVALID_ARG, "workspace must be set");
  if (!aligned(ws, 256)) return fail(VT_ERR_MISALIGNED, "workspace must be 256-byte aligned");
  if (have < need) return fail(VT_ERR_INVALID_ARG, "workspace holds %zu bytes, %zu needed", have, need);
  return VT_OK;
}

// Workspace of the ragged products: the status, the converted activations and, for the
// combining product, the pairs' outputs [pairs][N] in bf16.
constexpr size_t kActOff = 256;
inline int64_t scratch_ld(int64_t N) { return (N + 7) / 8 * 8; }
size_t act_end(vt_fp4_handle W, int64_t pairs) {
  return kActOff + up256(ragged_act_bytes(pairs, W->KT));
}

vt_status ragged(const void* A, int64_t lda, vt_fp4_handle W, const int32_t* order,
                 const int32_t* offsets, int64_t pairs, int64_t topk, int flags, void* C,
                 int64_t ldc, void* ws, size_t ws_bytes, vt_stream_t s,
                 const vt_fp4_gemm_opts* opts) {
  if (!W) return fail(VT_ERR_INVALID_ARG, "weight handle is NULL");
  if (opts && (opts->grid || opts->warps || opts->stages || opts->force_path ||
               opts->wait_limit_us < 0 || opts->withhold_weights == INT_MIN))
    return fail(VT_ERR_INVALID_ARG, "only wait_limit_us (>= 0) and withhold_weights may be set");
  if (vt_status st = check_groups(pairs, W->E)) return st;
  if (topk < 1 || topk > kMaxTopk) return fail(VT_ERR_INVALID_ARG, "topk must be in [1, %d]", kMaxTopk);
  if (pairs % topk) return fail(VT_ERR_INVALID_ARG, "pairs must be a multiple of topk");
  if (flags & ~(VT_RAGGED_GATHER | VT_RAGGED_SCATTER | VT_RAGGED_SILU_MUL))
    return fail(VT_ERR_INVALID_ARG, "unknown flags 0x%x", flags);
  const bool silu = flags & VT_RAGGED_SILU_MUL;
  if (silu != (W->layout == (int)kLayoutPaired))
    return fail(VT_ERR_INVALID_ARG,
                "the SiLU-and-multiply epilogue goes with a weight packed as paired gate and up");
  if (pairs == 0) return VT_OK;
  if (!A || !C || !order || !offsets)
    return fail(VT_ERR_INVALID_ARG, "A, C, order and offsets must be set");
  const int64_t cols = silu ? W->seg_split : W->N;
  if (lda < W->K || ldc < cols)
    return fail(VT_ERR_INVALID_ARG, "lda (%lld) must be >= K and ldc (%lld) >= the output columns",
                (long long)lda, (long long)ldc);
  if (!aligned(A, 16) || lda % 8)
    return fail(VT_ERR_MISALIGNED, "A must be 16-byte aligned with lda %% 8 == 0");
  if (!aligned(C, 2)) return fail(VT_ERR_MISALIGNED, "C must be 2-byte aligned");
  if (!aligned(order, 4) || !aligned(offsets, 4))
    return fail(VT_ERR_MISALIGNED, "order and offsets must be 4-byte aligned");
  if (vt_status st = check_workspace(ws, ws_bytes, act_end(W, pairs))) return st;
  RaggedLaunch L;
  L.packed = W->packed;
  L.fmt = W->fmt;
  L.N = W->N;
  L.K = W->K;
  L.RT = W->RT;
  L.KT = W->KT;
  L.seg_split = W->seg_split;
  L.layout = (uint32_t)W->layout;
  L.expert_bytes = W->expert_bytes;
  L.E = (int)W->E;
  L.A = A;
  L.lda = lda;
  L.order = order;
  L.offsets = offsets;
  L.pairs = pairs;
  L.topk = (int)topk;
  L.gather = (flags & VT_RAGGED_GATHER) ? 1 : 0;
  L.scatter = (flags & VT_RAGGED_SCATTER) ? 1 : 0;
  L.silu = silu ? 1 : 0;
  L.C = C;
  L.ldc = ldc;
  L.status = reinterpret_cast<int*>(ws);
  L.act = reinterpret_cast<uint8_t*>(ws) + kActOff;
  L.wait_ns = opts ? (uint64_t)opts->wait_limit_us * 1000ull : 0;
  L.withhold = opts ? opts->withhold_weights : 0;
  RaggedShape shape = {};
  if (vt_status st = done(launch_ragged(L, (cudaStream_t)s, &shape), "ragged product launch")) return st;
  W->info.path = 4;
  W->info.tile_epilogue = 0;
  W->info.stage_k_tiles = 1;
  W->info.grid = shape.grid;
  W->info.warps_per_cta = shape.warps;
  W->info.m_tile = shape.tokens;
  W->info.items = shape.items;
  W->info.launches = 2;  // the activation pre-pass and the product
  W->info.calls += 1;
  return VT_OK;
}

}  // namespace

extern "C" {

vt_status vt_fp4_group_workspace_bytes(int64_t pairs, int64_t E, size_t* bytes) {
  if (!bytes) return fail(VT_ERR_INVALID_ARG, "bytes is NULL");
  if (vt_status st = check_groups(pairs, E)) return st;
  *bytes = route_workspace_bytes(pairs, E);
  return VT_OK;
}

vt_status vt_fp4_group_rows(const int32_t* ids, int64_t pairs, int64_t E, int32_t* order,
                            int32_t* offsets, void* workspace, size_t ws_bytes, vt_stream_t s) {
  if (vt_status st = check_groups(pairs, E)) return st;
  if (!offsets || (pairs && (!ids || !order)))
    return fail(VT_ERR_INVALID_ARG, "ids, order and offsets must be set");
  if (!aligned(ids, 4) || !aligned(order, 4) || !aligned(offsets, 4))
    return fail(VT_ERR_MISALIGNED, "ids, order and offsets must be 4-byte aligned");
  if (vt_status st = check_workspace(workspace, ws_bytes, route_workspace_bytes(pairs, E))) return st;
  RouteLaunch L = {};
  L.M = pairs;
  L.E = (int)E;
  L.topk = 1;
  L.ids = const_cast<int32_t*>(ids);
  L.order = order;
  L.offsets = offsets;
  L.workspace = workspace;
  return done(launch_route(L, (cudaStream_t)s), "grouping launch");
}

vt_status vt_fp4_moe_route(const void* logits, int logits_bf16, int64_t M, int64_t ld, int64_t E,
                           int64_t topk, int scoring, const float* bias, int renormalize,
                           float scale, int32_t* ids, float* weights, int32_t* order,
                           int32_t* offsets, void* workspace, size_t ws_bytes, vt_stream_t s) {
  if (M < 0 || M >= kMaxPairs) return fail(VT_ERR_INVALID_ARG, "M must be in [0, 2^31 - 2^27)");
  if (topk < 1 || topk > kMaxTopk) return fail(VT_ERR_INVALID_ARG, "topk must be in [1, %d]", kMaxTopk);
  if (vt_status st = check_groups(M * topk, E)) return st;
  if (topk > E) return fail(VT_ERR_INVALID_ARG, "topk (%lld) exceeds E (%lld)", (long long)topk, (long long)E);
  if (logits_bf16 != 0 && logits_bf16 != 1)
    return fail(VT_ERR_INVALID_ARG, "logits_bf16 must be 0 (fp32) or 1 (bf16)");
  if (scoring != 0 && scoring != 1) return fail(VT_ERR_INVALID_ARG, "scoring must be 0 or 1");
  if (bias && scoring != 1) return fail(VT_ERR_INVALID_ARG, "a bias goes with scoring 1 (sigmoid)");
  if (!isfinite(scale)) return fail(VT_ERR_INVALID_ARG, "scale must be finite");
  if (!offsets || (M && (!logits || !ids || !weights || !order)))
    return fail(VT_ERR_INVALID_ARG, "logits, ids, weights, order and offsets must be set");
  if (ld < E) return fail(VT_ERR_INVALID_ARG, "ld (%lld) must be >= E", (long long)ld);
  if (!aligned(logits, logits_bf16 ? 2 : 4) || !aligned(bias, 4) || !aligned(ids, 4) ||
      !aligned(weights, 4) || !aligned(order, 4) || !aligned(offsets, 4))
    return fail(VT_ERR_MISALIGNED, "every pointer must be aligned to its type");
  if (vt_status st = check_workspace(workspace, ws_bytes, route_workspace_bytes(M * topk, E))) return st;
  RouteLaunch L;
  L.logits = logits;
  L.bf16 = logits_bf16;
  L.ld = ld;
  L.scoring = scoring;
  L.bias = bias;
  L.renormalize = renormalize ? 1 : 0;
  L.scale = scale;
  L.M = M;
  L.E = (int)E;
  L.topk = (int)topk;
  L.ids = ids;
  L.weights = weights;
  L.order = order;
  L.offsets = offsets;
  L.workspace = workspace;
  return done(launch_route(L, (cudaStream_t)s), "router launch");
}

vt_status vt_fp4_ragged_workspace_bytes(vt_fp4_handle W, int64_t M_max, int64_t topk,
                                        size_t* bytes) {
  if (!W) return fail(VT_ERR_INVALID_ARG, "weight handle is NULL");
  if (!bytes) return fail(VT_ERR_INVALID_ARG, "bytes is NULL");
  if (topk < 1 || topk > kMaxTopk) return fail(VT_ERR_INVALID_ARG, "topk must be in [1, %d]", kMaxTopk);
  if (M_max < 0 || M_max >= kMaxPairs) return fail(VT_ERR_INVALID_ARG, "M_max must be in [0, 2^31 - 2^27)");
  if (vt_status st = check_groups(M_max * topk, W->E)) return st;
  // a paired weight's output is the caller's; only the combining product keeps scratch
  const size_t scratch = W->layout == (int)kLayoutPaired ? 0 : (size_t)(M_max * topk) * scratch_ld(W->N) * 2;
  *bytes = act_end(W, M_max * topk) + up256(scratch);
  return VT_OK;
}

vt_status vt_fp4_w4a16_gemm_ragged(const void* A, int64_t lda, vt_fp4_handle W,
                                   const int32_t* order, const int32_t* offsets, int64_t pairs,
                                   int64_t topk, int flags, void* C, int64_t ldc, void* workspace,
                                   size_t ws_bytes, vt_stream_t s) {
  return vt_fp4_w4a16_gemm_ragged_ex(A, lda, W, order, offsets, pairs, topk, flags, C, ldc, workspace,
                                     ws_bytes, s, nullptr);
}

vt_status vt_fp4_w4a16_gemm_ragged_ex(const void* A, int64_t lda, vt_fp4_handle W,
                                      const int32_t* order, const int32_t* offsets, int64_t pairs,
                                      int64_t topk, int flags, void* C, int64_t ldc,
                                      void* workspace, size_t ws_bytes, vt_stream_t s,
                                      const vt_fp4_gemm_opts* opts) {
  return ragged(A, lda, W, order, offsets, pairs, topk, flags, C, ldc, workspace, ws_bytes, s, opts);
}

vt_status vt_fp4_w4a16_gemm_ragged_combine(const void* A, int64_t lda, vt_fp4_handle W,
                                           const int32_t* ids, const int32_t* order,
                                           const int32_t* offsets, const float* weights,
                                           int64_t M, int64_t topk, void* C, int64_t ldc,
                                           void* workspace, size_t ws_bytes, vt_stream_t s) {
  if (M < 0 || M >= kMaxPairs) return fail(VT_ERR_INVALID_ARG, "M must be in [0, 2^31 - 2^27)");
  size_t need = 0;
  if (vt_status st = vt_fp4_ragged_workspace_bytes(W, M, topk, &need)) return st;
  if (W->layout != (int)kLayoutRows)
    return fail(VT_ERR_INVALID_ARG, "the combining product takes a plain grouped weight");
  if (M == 0) return VT_OK;
  if (!ids || !weights || !C) return fail(VT_ERR_INVALID_ARG, "ids, weights and C must be set");
  if (!aligned(ids, 4) || !aligned(weights, 4))
    return fail(VT_ERR_MISALIGNED, "ids and weights must be 4-byte aligned");
  if (ldc < W->N) return fail(VT_ERR_INVALID_ARG, "ldc (%lld) must be >= N", (long long)ldc);
  if (!aligned(C, 2)) return fail(VT_ERR_MISALIGNED, "C must be 2-byte aligned");
  if (vt_status st = check_workspace(workspace, ws_bytes, need)) return st;
  void* D = reinterpret_cast<uint8_t*>(workspace) + act_end(W, M * topk);
  const int64_t ldd = scratch_ld(W->N);
  if (vt_status st = ragged(A, lda, W, order, offsets, M * topk, topk, VT_RAGGED_SCATTER, D, ldd,
                            workspace, ws_bytes, s, nullptr))
    return st;
  if (vt_status st = done(launch_combine(D, M, (int)topk, W->N, ldd, ids, (int)W->E, weights, C, ldc,
                                         (cudaStream_t)s),
                          "combine launch"))
    return st;
  W->info.launches += 1;
  return VT_OK;
}

vt_status vt_fp4_lora_add(const void* x, int64_t M, int64_t ldx, int64_t K, const void* A,
                          const void* B, const float* scale, const int32_t* ranks, int64_t L,
                          int64_t R, int64_t N, const int32_t* order, const int32_t* offsets,
                          const void* y, int64_t ldy, void* out, int64_t ldo, vt_stream_t s) {
  if (L < 1 || L > kMaxGroups) return fail(VT_ERR_INVALID_ARG, "L must be in [1, %d]", kMaxGroups);
  if (R < 1 || R > kMaxRank) return fail(VT_ERR_INVALID_ARG, "R must be in [1, %d]", kMaxRank);
  if (M < 0 || M >= kMaxPairs) return fail(VT_ERR_INVALID_ARG, "M must be in [0, 2^31 - 2^27)");
  if (K < 1 || N < 1 || K > (int64_t)1 << 24 || N > (int64_t)1 << 24)
    return fail(VT_ERR_INVALID_ARG, "K and N must be in [1, 2^24]");
  if (ldx < K || ldy < N || ldo < N)
    return fail(VT_ERR_INVALID_ARG, "ldx must be >= K, ldy and ldo >= N");
  if (M == 0) return VT_OK;
  if (!x || !A || !B || !scale || !order || !offsets || !y || !out)
    return fail(VT_ERR_INVALID_ARG, "x, A, B, scale, order, offsets, y and out must be set");
  if (!aligned(x, 2) || !aligned(A, 2) || !aligned(B, 2) || !aligned(y, 2) || !aligned(out, 2) ||
      !aligned(scale, 4) || !aligned(ranks, 4) || !aligned(order, 4) || !aligned(offsets, 4))
    return fail(VT_ERR_MISALIGNED, "every pointer must be aligned to its type");
  if (y == out && ldy != ldo) return fail(VT_ERR_INVALID_ARG, "out == y needs ldo == ldy");
  LoraLaunch P;
  P.x = x;
  P.M = M;
  P.ldx = ldx;
  P.K = K;
  P.A = A;
  P.B = B;
  P.scale = scale;
  P.ranks = ranks;
  P.L = (int)L;
  P.R = (int)R;
  P.N = N;
  P.order = order;
  P.offsets = offsets;
  P.y = y;
  P.ldy = ldy;
  P.out = out;
  P.ldo = ldo;
  return done(launch_lora(P, (cudaStream_t)s), "adapter launch");
}

}  // extern "C"
