// C entry points of what a decoder layer runs between its products (declared in include/vt_fp4.h):
// the paged NVFP4 cache, the attention over it and the norms around the blocks.  Argument checks run
// before any CUDA call.
#include <limits.h>
#include <math.h>
#include <stdarg.h>
#include <stdio.h>

#include <atomic>

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

std::atomic<int> g_wait_us{0}, g_withhold{0};  // vt_fp4_attention_test_hooks

inline bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }
constexpr int64_t kMaxRows = (int64_t)1 << 24;       // tokens of a call
constexpr int64_t kMaxStride = (int64_t)1 << 32;     // elements between two rows
constexpr int64_t kMaxHeads = 1024;

vt_status check_page(int64_t page_size, int64_t heads, int64_t head_dim) {
  if (page_size != 16 && page_size != 32 && page_size != 64 && page_size != 128 && page_size != 256)
    return fail(VT_ERR_INVALID_ARG, "page_size must be 16, 32, 64, 128 or 256 (got %lld)", (long long)page_size);
  if (heads < 1 || heads > kMaxHeads) return fail(VT_ERR_INVALID_ARG, "heads must be in [1, %lld]", (long long)kMaxHeads);
  if (head_dim != 64 && head_dim != 128 && head_dim != 256)
    return fail(VT_ERR_UNSUPPORTED, "head_dim must be 64, 128 or 256 (got %lld)", (long long)head_dim);
  return VT_OK;
}

int64_t page_bytes(int64_t page_size, int64_t heads, int64_t head_dim) {
  return heads * (page_size / kKvTile) * kv_tile_bytes((int)head_dim);
}

vt_status check_cache(const vt_fp4_kv_cache* c, KvCache* out) {
  if (!c) return fail(VT_ERR_INVALID_ARG, "the cache is NULL");
  if (vt_status st = check_page(c->page_size, c->heads, c->head_dim)) return st;
  if (c->pages < 1 || c->pages >= ((int64_t)1 << 31) / c->page_size)
    return fail(VT_ERR_INVALID_ARG, "pages must be at least 1 and pages * page_size below 2^31");
  if (c->page_stride < page_bytes(c->page_size, c->heads, c->head_dim) || c->page_stride > kMaxStride)
    return fail(VT_ERR_INVALID_ARG, "page_stride (%lld) must be in [%lld, 2^32]", (long long)c->page_stride,
                (long long)page_bytes(c->page_size, c->heads, c->head_dim));
  if (!c->data || !c->k_scale || !c->v_scale)
    return fail(VT_ERR_INVALID_ARG, "the cache's data, k_scale and v_scale must be set");
  if (!aligned(c->data, 128) || c->page_stride % 128)
    return fail(VT_ERR_MISALIGNED, "the cache's data and page_stride must be multiples of 128 bytes");
  if (!aligned(c->k_scale, 4) || !aligned(c->v_scale, 4))
    return fail(VT_ERR_MISALIGNED, "k_scale and v_scale must be 4-byte aligned");
  out->data = reinterpret_cast<uint8_t*>(c->data);
  out->page_stride = c->page_stride;
  out->slots = c->pages * c->page_size;
  out->pages = (int)c->pages;
  out->heads = (int)c->heads;
  out->page_size = (int)c->page_size;
  out->page_shift = __builtin_ctz((unsigned)c->page_size);
  out->k_scale = c->k_scale;
  out->v_scale = c->v_scale;
  return VT_OK;
}

vt_status check_rows(int64_t T) {
  if (T < 0 || T > kMaxRows) return fail(VT_ERR_INVALID_ARG, "T must be in [0, 2^24] (got %lld)", (long long)T);
  return VT_OK;
}

// A matrix of bf16 rows that the kernels take 16 bytes at a time.
vt_status check_heads(const void* p, int64_t ld, int64_t cols, const char* name) {
  if (!p) return fail(VT_ERR_INVALID_ARG, "%s must be set", name);
  if (ld < cols || ld > kMaxStride)
    return fail(VT_ERR_INVALID_ARG, "the row stride of %s (%lld) must be in [%lld, 2^32]", name, (long long)ld, (long long)cols);
  if (!aligned(p, 16) || ld % 8)
    return fail(VT_ERR_MISALIGNED, "%s must be 16-byte aligned with a row stride that is a multiple of 8", name);
  return VT_OK;
}

vt_status check_q_heads(int64_t q_heads, int64_t heads) {
  if (q_heads < 1 || q_heads % heads || q_heads / heads > kMaxGroupHeads)
    return fail(VT_ERR_INVALID_ARG, "q_heads (%lld) must be a multiple of the cache's heads (%lld), at most %d times",
                (long long)q_heads, (long long)heads, kMaxGroupHeads);
  return VT_OK;
}

vt_status move(const vt_fp4_kv_cache* cache, int64_t T, const int64_t* slots, uint8_t* kc, uint8_t* ks,
               uint8_t* vc, uint8_t* vs, void* k, void* v, int dir, vt_stream_t s) {
  KvMoveLaunch L = {};
  if (vt_status st = check_cache(cache, &L.cache)) return st;
  if (vt_status st = check_rows(T)) return st;
  if (T == 0) return VT_OK;
  if (!slots || (dir == 2 ? !k || !v : !kc || !ks || !vc || !vs))
    return fail(VT_ERR_INVALID_ARG, "slots and the tokens' buffers must be set");
  if (!aligned(slots, 8) || !aligned(kc, 8) || !aligned(vc, 8) || !aligned(k, 16) || !aligned(v, 16))
    return fail(VT_ERR_MISALIGNED, "slots and codes must be 8-byte aligned, k and v 16-byte aligned");
  L.T = T;
  L.slots = slots;
  L.k_codes = kc;
  L.k_scales = ks;
  L.v_codes = vc;
  L.v_scales = vs;
  L.k = k;
  L.v = v;
  return done(launch_kv_move(L, (int)cache->head_dim, dir, (cudaStream_t)s), "cache launch");
}

}  // namespace

extern "C" {

vt_status vt_fp4_kv_page_bytes(int64_t page_size, int64_t heads, int64_t head_dim, size_t* bytes) {
  if (!bytes) return fail(VT_ERR_INVALID_ARG, "bytes is NULL");
  if (vt_status st = check_page(page_size, heads, head_dim)) return st;
  *bytes = (size_t)page_bytes(page_size, heads, head_dim);
  return VT_OK;
}

vt_status vt_fp4_kv_append(const vt_fp4_kv_cache* cache, int64_t T, const void* q, int64_t q_heads,
                           int64_t ldq, const void* k, int64_t ldk, const void* v, int64_t ldv,
                           const int64_t* slots, const int32_t* positions, const float* table,
                           int64_t table_rows, int64_t rot, int interleaved, const void* q_norm,
                           const void* k_norm, int norms_fp32, float eps, void* q_out, int64_t ldo,
                           vt_stream_t s) {
  AppendLaunch L = {};
  if (vt_status st = check_cache(cache, &L.cache)) return st;
  if (vt_status st = check_rows(T)) return st;
  const int64_t D = cache->head_dim;
  if (q) {
    if (vt_status st = check_q_heads(q_heads, cache->heads)) return st;
  } else if (q_heads || q_norm || q_out) {
    return fail(VT_ERR_INVALID_ARG, "without q there are no q_heads, q_norm and q_out");
  }
  if (rot < 0 || rot > D || rot % 16)
    return fail(VT_ERR_INVALID_ARG, "rot must be a multiple of 16 in [0, head_dim] (got %lld)", (long long)rot);
  if (rot ? !positions || !table : positions || table)
    return fail(VT_ERR_INVALID_ARG, "positions and table go with rot > 0");
  if (rot && (table_rows < 1 || table_rows > ((int64_t)1 << 31) - 1))
    return fail(VT_ERR_INVALID_ARG, "table_rows must be in [1, 2^31 - 1]");
  if (interleaved != 0 && interleaved != 1) return fail(VT_ERR_INVALID_ARG, "interleaved must be 0 or 1");
  if (norms_fp32 != 0 && norms_fp32 != 1)
    return fail(VT_ERR_INVALID_ARG, "norms_fp32 must be 0 (bf16) or 1 (fp32)");
  if (q && !q_norm != !k_norm) return fail(VT_ERR_INVALID_ARG, "q_norm and k_norm go together");
  if (k_norm && !(eps >= 0.0f && isfinite(eps))) return fail(VT_ERR_INVALID_ARG, "eps must be finite and not negative");
  if (T == 0) return VT_OK;
  if (q) {
    if (vt_status st = check_heads(q, ldq, q_heads * D, "q")) return st;
    if (vt_status st = check_heads(q_out, ldo, q_heads * D, "q_out")) return st;
    if (q == q_out && ldq != ldo) return fail(VT_ERR_INVALID_ARG, "q_out == q needs ldo == ldq");
  }
  if (vt_status st = check_heads(k, ldk, cache->heads * D, "k")) return st;
  if (vt_status st = check_heads(v, ldv, cache->heads * D, "v")) return st;
  if (!slots) return fail(VT_ERR_INVALID_ARG, "slots must be set");
  if (!aligned(slots, 8) || !aligned(positions, 4) || !aligned(table, 16) || !aligned(q_norm, 16) || !aligned(k_norm, 16))
    return fail(VT_ERR_MISALIGNED, "slots must be 8-byte, positions 4-byte, table and norms 16-byte aligned");
  L.T = T;
  L.q = q;
  L.q_heads = (int)q_heads;
  L.ldq = ldq;
  L.k = k;
  L.ldk = ldk;
  L.v = v;
  L.ldv = ldv;
  L.slots = slots;
  L.positions = positions;
  L.table = table;
  L.table_rows = table_rows;
  L.rot = (int)rot;
  L.interleaved = interleaved;
  L.q_norm = q_norm;
  L.k_norm = k_norm;
  L.norms_fp32 = norms_fp32;
  L.eps = eps;
  L.q_out = q_out;
  L.ldo = ldo;
  return done(launch_append(L, (int)D, (cudaStream_t)s), "append launch");
}

vt_status vt_fp4_kv_read(const vt_fp4_kv_cache* cache, int64_t T, const int64_t* slots, void* k, void* v,
                         vt_stream_t s) {
  return move(cache, T, slots, nullptr, nullptr, nullptr, nullptr, k, v, 2, s);
}

vt_status vt_fp4_kv_put(const vt_fp4_kv_cache* cache, int64_t T, const int64_t* slots,
                        const uint8_t* k_codes, const uint8_t* k_scales, const uint8_t* v_codes,
                        const uint8_t* v_scales, vt_stream_t s) {
  return move(cache, T, slots, const_cast<uint8_t*>(k_codes), const_cast<uint8_t*>(k_scales),
              const_cast<uint8_t*>(v_codes), const_cast<uint8_t*>(v_scales), nullptr, nullptr, 0, s);
}

vt_status vt_fp4_kv_get(const vt_fp4_kv_cache* cache, int64_t T, const int64_t* slots, uint8_t* k_codes,
                        uint8_t* k_scales, uint8_t* v_codes, uint8_t* v_scales, vt_stream_t s) {
  return move(cache, T, slots, k_codes, k_scales, v_codes, v_scales, nullptr, nullptr, 1, s);
}

vt_status vt_fp4_attention_workspace_bytes(const vt_fp4_kv_cache* cache, int64_t T_max, int64_t B_max,
                                           int64_t q_heads, size_t* bytes) {
  if (!bytes) return fail(VT_ERR_INVALID_ARG, "bytes is NULL");
  KvCache c;
  if (vt_status st = check_cache(cache, &c)) return st;
  if (vt_status st = check_rows(T_max)) return st;
  if (vt_status st = check_rows(B_max)) return st;
  if (vt_status st = check_q_heads(q_heads, cache->heads)) return st;
  *bytes = attend_workspace_bytes(T_max, (int)(q_heads / cache->heads), (int)cache->head_dim);
  return VT_OK;
}

vt_status vt_fp4_paged_attention(const vt_fp4_kv_cache* cache, int64_t T, const void* q, int64_t q_heads,
                                 int64_t ldq, const int32_t* tables, int64_t ldt, const int32_t* lens,
                                 const int32_t* starts, int64_t B, float scale, int64_t window,
                                 const float* sinks, void* out, int64_t ldo, void* workspace,
                                 size_t ws_bytes, vt_stream_t s) {
  AttendLaunch L = {};
  if (vt_status st = check_cache(cache, &L.cache)) return st;
  if (vt_status st = check_rows(T)) return st;
  if (B < 0 || B > kMaxRows) return fail(VT_ERR_INVALID_ARG, "B must be in [0, 2^24] (got %lld)", (long long)B);
  if (vt_status st = check_q_heads(q_heads, cache->heads)) return st;
  if (!starts && T != B) return fail(VT_ERR_INVALID_ARG, "without starts there is one row per sequence: T must be B");
  if (!isfinite(scale)) return fail(VT_ERR_INVALID_ARG, "scale must be finite");
  if (window < 0) return fail(VT_ERR_INVALID_ARG, "window must not be negative");
  if (ldt < 1 || ldt > ((int64_t)1 << 30) / cache->page_size)
    return fail(VT_ERR_INVALID_ARG, "ldt must be at least 1 and ldt * page_size at most 2^30");
  if (T == 0 || B == 0) return VT_OK;
  if (vt_status st = check_heads(q, ldq, q_heads * cache->head_dim, "q")) return st;
  if (vt_status st = check_heads(out, ldo, q_heads * cache->head_dim, "out")) return st;
  if (q == out && ldq != ldo) return fail(VT_ERR_INVALID_ARG, "out == q needs ldo == ldq");
  if (!tables || !lens) return fail(VT_ERR_INVALID_ARG, "tables and lens must be set");
  if (!aligned(tables, 4) || !aligned(lens, 4) || !aligned(starts, 4) || !aligned(sinks, 4))
    return fail(VT_ERR_MISALIGNED, "tables, lens, starts and sinks must be 4-byte aligned");
  const size_t need = attend_workspace_bytes(starts ? T : 0, (int)(q_heads / cache->heads), (int)cache->head_dim);
  if (!workspace) return fail(VT_ERR_INVALID_ARG, "workspace must be set");
  if (!aligned(workspace, 256)) return fail(VT_ERR_MISALIGNED, "workspace must be 256-byte aligned");
  if (ws_bytes < need) return fail(VT_ERR_INVALID_ARG, "workspace holds %zu bytes, %zu needed", ws_bytes, need);
  L.T = T;
  L.q = q;
  L.ldq = ldq;
  L.q_heads = (int)q_heads;
  L.group = (int)(q_heads / cache->heads);
  L.tables = tables;
  L.ldt = ldt;
  L.lens = lens;
  L.starts = starts;
  L.B = B;
  L.scale = scale;
  L.window = window;
  L.sinks = sinks;
  L.out = out;
  L.ldo = ldo;
  L.workspace = reinterpret_cast<uint8_t*>(workspace);
  L.wait_ns = (uint64_t)g_wait_us.load() * 1000ull;
  L.withhold = g_withhold.load();
  return done(launch_attend(L, (int)cache->head_dim, (cudaStream_t)s), "attention launch");
}

vt_status vt_fp4_attention_test_hooks(int wait_limit_us, int withhold) {
  if (wait_limit_us < 0 || withhold == INT_MIN)
    return fail(VT_ERR_INVALID_ARG, "wait_limit_us must be >= 0, withhold above INT_MIN");
  g_wait_us.store(wait_limit_us);
  g_withhold.store(withhold);
  return VT_OK;
}

vt_status vt_fp4_residual_norm(const void* x, int64_t T, int64_t H, int64_t ldx, const void* residual,
                               int64_t ldr, int residual_fp32, const void* post_weight, const void* gate,
                               int64_t ldg, float scale, const void* weight, int weights_fp32,
                               float eps, void* h, int64_t ldh, void* y, int64_t ldy, vt_stream_t s) {
  if (vt_status st = check_rows(T)) return st;
  if (H < 1 || H > kMaxNormWidth) return fail(VT_ERR_INVALID_ARG, "H must be in [1, %d]", kMaxNormWidth);
  if (residual_fp32 != 0 && residual_fp32 != 1)
    return fail(VT_ERR_INVALID_ARG, "residual_fp32 must be 0 (bf16) or 1 (fp32)");
  if (weights_fp32 != 0 && weights_fp32 != 1)
    return fail(VT_ERR_INVALID_ARG, "weights_fp32 must be 0 (bf16) or 1 (fp32)");
  if (!isfinite(scale)) return fail(VT_ERR_INVALID_ARG, "scale must be finite");
  if (!(eps >= 0.0f && isfinite(eps))) return fail(VT_ERR_INVALID_ARG, "eps must be finite and not negative");
  if (!residual != !h) return fail(VT_ERR_INVALID_ARG, "residual and h go together");
  if (T == 0) return VT_OK;
  if (!x || !weight || !y) return fail(VT_ERR_INVALID_ARG, "x, weight and y must be set");
  const int64_t lds[] = {ldx, ldy, residual ? ldr : H, residual ? ldh : H, gate && ldg ? ldg : H};
  for (int64_t ld : lds)
    if (ld < H || ld > kMaxStride) return fail(VT_ERR_INVALID_ARG, "every row stride must be in [H, 2^32] (got %lld)", (long long)ld);
  const size_t r = residual_fp32 ? 4 : 2, w = weights_fp32 ? 4 : 2;
  if (!aligned(x, 2) || !aligned(y, 2) || !aligned(gate, 2) || !aligned(residual, r) || !aligned(h, r) ||
      !aligned(weight, w) || !aligned(post_weight, w))
    return fail(VT_ERR_MISALIGNED, "every pointer must be aligned to its type");
  if (h && h == residual && ldh != ldr) return fail(VT_ERR_INVALID_ARG, "h == residual needs ldh == ldr");
  if (x == y && ldx != ldy) return fail(VT_ERR_INVALID_ARG, "y == x needs ldy == ldx");
  NormLaunch L = {};
  L.x = x;
  L.T = T;
  L.H = H;
  L.ldx = ldx;
  L.residual = residual;
  L.ldr = ldr;
  L.residual_fp32 = residual_fp32;
  L.post_weight = post_weight;
  L.gate = gate;
  L.ldg = ldg;
  L.scale = scale;
  L.weight = weight;
  L.weights_fp32 = weights_fp32;
  L.eps = eps;
  L.h = h;
  L.ldh = ldh;
  L.y = y;
  L.ldy = ldy;
  return done(launch_norm(L, (cudaStream_t)s), "norm launch");
}

}  // extern "C"
