// Causal attention over the paged NVFP4 cache.  One warp per (row, head), the keys one after another,
// with the running maximum and sum of the softmax.
#include <cuda_bf16.h>

#include "actq.cuh"
#include "attend.cuh"
#include "common.cuh"
#include "kernels.h"
#include "kv.cuh"

namespace vt {

namespace {

template <int D>
__global__ void __launch_bounds__(128) k_attend_simple(const AttendLaunch p) {
  constexpr int PER = D / 32;
  const int lane = threadIdx.x & 31;
  const int64_t w = blockIdx.x * 4ll + (threadIdx.x >> 5);
  if (w >= p.T * p.q_heads) return;
  const int64_t t = w / p.q_heads;
  const int h = (int)(w - t * p.q_heads), kvh = h / p.group;
  int64_t b = t, first = t, n = 1;
  if (p.starts) {
    int64_t lo = 0, hi = p.B;  // the last sequence that starts at or before t
    while (hi - lo > 1) {
      const int64_t mid = (lo + hi) / 2;
      if (p.starts[mid] <= t) lo = mid;
      else hi = mid;
    }
    b = lo;
    // an empty sequence shares its start with the next: lo is the last of them
    first = p.starts[b];
    n = p.starts[b + 1] - first;
    if (t < first || t >= first + n) return;
  }
  int64_t len = p.lens[b];
  const int64_t most = p.ldt * p.cache.page_size;
  len = len < 0 ? 0 : len > most ? most : len;
  const int64_t pos = len - n + (t - first);
  int64_t j0 = p.window > 0 ? pos - p.window + 1 : 0;
  if (j0 < 0) j0 = 0;
  float q[PER], o[PER], m = -INFINITY, l = 0.0f;
  const __nv_bfloat16* qp = reinterpret_cast<const __nv_bfloat16*>(p.q) + t * p.ldq + (int64_t)h * D + lane * PER;
  for (int i = 0; i < PER; ++i) q[i] = __bfloat162float(qp[i]), o[i] = 0.0f;
  bool any = false;
  const float ks = p.cache.k_scale[kvh], vs = p.cache.v_scale[kvh];
  for (int64_t j = j0; j <= pos; ++j) {
    const int64_t page = p.tables[b * p.ldt + (j >> p.cache.page_shift)];
    if (page < 0 || page >= p.cache.pages) continue;
    any = true;
    const int in = (int)(j & (p.cache.page_size - 1)), r = in % kKvTile;
    const uint8_t* tile = kv_tile<D>(p.cache, page, kvh, in);
    const int d = lane * PER;
    auto values = [&](bool v, float (&x)[PER]) {
      const uint32_t sb = tile[v ? kv_v_scale(D, r, d / 16) : kv_k_scale(D, r, d / 16)];
      const float step = __half2float(__ushort_as_half((unsigned short)e4m3x2_to_f16x2(sb)));
      for (int i = 0; i < PER; i += 2) {
        const uint32_t f = e2m1x2_to_f16x2(tile[v ? kv_v_code(D, r, (d + i) / 2) : kv_k_code(D, r, (d + i) / 2)]);
        const float2 c = __half22float2(bits_h2(f));
        x[i] = c.x * step;
        x[i + 1] = c.y * step;
      }
    };
    float x[PER], s = 0.0f;
    values(false, x);
    for (int i = 0; i < PER; ++i) s += q[i] * x[i];
    for (int k = 16; k; k >>= 1) s += __shfl_xor_sync(0xffffffffu, s, k);
    s *= ks * p.scale;
    const float mn = s > m ? s : m;
    const float a = m == -INFINITY ? 0.0f : expf(m - mn), e = expf(s - mn);
    m = mn;
    l = l * a + e;
    values(true, x);
    for (int i = 0; i < PER; ++i) o[i] = o[i] * a + e * x[i];
  }
  if (p.sinks && any) {
    const float sk = p.sinks[h], mn = fmaxf(sk, m), a = expf(m - mn);
    l = l * a + expf(sk - mn);
    for (int i = 0; i < PER; ++i) o[i] *= a;
  }
  __nv_bfloat16* op = reinterpret_cast<__nv_bfloat16*>(p.out) + t * p.ldo + (int64_t)h * D + lane * PER;
  for (int i = 0; i < PER; ++i) op[i] = __float2bfloat16(any ? o[i] * vs / l : 0.0f);
}

}  // namespace

size_t attend_workspace_bytes(int64_t T, int64_t B, int q_heads, int heads, int head_dim) {
  return kAttendCleared + attend_row_parts_bytes(head_dim);
}

cudaError_t launch_attend(const AttendLaunch& L, int head_dim, cudaStream_t s) {
  if (!L.starts) return launch_attend_row(L, head_dim, s);
  const unsigned blocks = (unsigned)((L.T * L.q_heads + 3) / 4);
  if (head_dim == 64) k_attend_simple<64><<<blocks, 128, 0, s>>>(L);
  else if (head_dim == 128) k_attend_simple<128><<<blocks, 128, 0, s>>>(L);
  else k_attend_simple<256><<<blocks, 128, 0, s>>>(L);
  return cudaGetLastError();
}

}  // namespace vt
