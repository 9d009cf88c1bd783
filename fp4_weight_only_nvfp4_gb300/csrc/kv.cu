// The paged NVFP4 cache: appending tokens (per-head norm, rotation and quantisation on the way),
// reading values back, and moving raw tokens in and out.
#include <cuda_bf16.h>

#include "actq.cuh"
#include "common.cuh"
#include "kernels.h"
#include "kv.cuh"

namespace vt {

namespace {

constexpr int kAppendThreads = 256;

__device__ __forceinline__ void unpack8(const uint4 v, float (&x)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    x[2 * q] = bf16_lo(w[q]);
    x[2 * q + 1] = bf16_hi(w[q]);
  }
}

__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * q], x[2 * q + 1]);
    w[q] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ void load_norm8(const void* w, int fp32, int d, float (&x)[8]) {
  if (fp32) {
    const float4* p = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(w) + d);
    const float4 a = p[0], b = p[1];
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  } else {
    unpack8(*reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(w) + d), x);
  }
}

// Largest magnitude pattern (sign cleared) among 8 bf16 values.
__device__ __forceinline__ uint32_t magnitude8(const uint4 v) {
  constexpr uint32_t M = 0x7FFF7FFFu;
  const uint32_t m = __vmaxu2(__vmaxu2(v.x & M, v.y & M), __vmaxu2(v.z & M, v.w & M));
  return max(m & 0xFFFFu, m >> 16);
}

// Sum of a vector's squares over its LANES lanes (8 bf16 values each), rounded to fp32 once.  The
// values are taken times 2^-e, e the exponent of the largest (mag: its pattern), so that a square x^2
// is below 4 and has 16 bits; it is cut at 2^-13 into a + b, a = (x^2 + C) - C.  256 a's add up without
// a rounding (below 2^24 units of 2^-13), the b's with errors of 2^-23 of what is below 2^-6 (a lane's) and 2^-37 a lane: the
// sum is held to 2^-32 of the largest square.  Where a vector takes the whole warp its lanes add integers, one instruction for
// the ten of a sum by shuffles (8192 tokens of 32 heads of 256, read back: 99 us with shuffles and one value at a time, 98 with two at a
// time, 91 so).
// Every lane of the warp is in the sums over the lanes, whatever its vector holds: where the warp has several vectors,
// one with an inf or NaN gets that in the place of its sum at the end, and no lane leaves before.
template <int LANES>
__device__ __forceinline__ float sum_squares(const float (&x)[8], uint32_t mag) {
  const bool finite = mag < 0x7F80u;
  const float special = __uint_as_float(mag << 16);  // inf or NaN
  if constexpr (LANES == 32) {
    if (!finite) return special;  // one vector, one mag: the whole warp
  }
  const int e = min(max((int)(mag >> 7) - 127, -126), 126);  // (at 2^127 the sum is inf in any case)
  const float down = pow2f(-e), up = pow2f(e);
  constexpr float C = 1.5f * 1024.0f;                      // its last bit is 2^-13
  const uint64_t down2 = pair(down, down), c2 = pair(C, C), minus = pair(-1.0f, -1.0f);
  uint64_t na = 0, ab = 0;                                 // -a, b
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    const uint64_t v = mul2(pair(x[i], x[i + 1]), down2);
    const uint64_t nt = fma2(fma2(v, v, c2), minus, c2);   // C - (x^2 + C)
    na = add2(na, nt);
    ab = add2(ab, fma2(v, v, nt));
  }
  float a0, a1, b0, b1;
  split(na, a0, a1);
  split(ab, b0, b1);
  float a = -__fadd_rn(a0, a1), b = __fadd_rn(b0, b1);
  if constexpr (LANES == 32) {  // a whole warp adds integers in one instruction: units of 2^-13 and of 2^-36
    a = (float)__reduce_add_sync(0xffffffffu, (int)(a * 8192.0f)) * (1.0f / 8192.0f);
    b = (float)__reduce_add_sync(0xffffffffu, __float2int_rn(b * 0x1p36f)) * 0x1p-36f;
  } else {
#pragma unroll
    for (int m = 1; m < LANES; m <<= 1) {
      a = __fadd_rn(a, __shfl_xor_sync(0xffffffffu, a, m));
      b = __fadd_rn(b, __shfl_xor_sync(0xffffffffu, b, m));
    }
  }
  return finite ? __fadd_rn(a, b) * up * up : special;
}

// Codes of x / d, each quotient rounded to fp32 first.  x times the rounded 1 / d is off by less than 2^-22 of
// the quotient, and the codes are monotone: where 2^-21 to both sides give the same ones, those are it.  Else, and
// where 1 / d has fewer bits, the quotients themselves (the append of 8192 tokens of 24 + 2 * 4 heads of 256: 82 us with divisions alone,
// 78 so, and 80 with a global of 1, where quotients of bf16 values meet borders often).
__device__ __forceinline__ uint32_t quotient_codes(const float (&x)[8], float d) {
  const float inv = __frcp_rn(d);
  const uint64_t less = pair(inv * (1.0f - 0x1p-21f), inv * (1.0f - 0x1p-21f)), more = pair(inv * (1.0f + 0x1p-21f), inv * (1.0f + 0x1p-21f));
  float lo[8], hi[8];
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    split(mul2(pair(x[i], x[i + 1]), less), lo[i], lo[i + 1]);
    split(mul2(pair(x[i], x[i + 1]), more), hi[i], hi[i + 1]);
  }
  uint32_t codes = aq_e2m1x8(lo);
  if (codes != aq_e2m1x8(hi) || !(d >= 0x1p-120f && d <= 0x1p120f)) {
#pragma unroll
    for (int i = 0; i < 8; ++i) lo[i] = __fdiv_rn(x[i], d);
    codes = aq_e2m1x8(lo);
  }
  return codes;
}

// D / 8 lanes take one head's vector of one token, 8 values each; a warp takes `steps` times 32 / (D /
// 8) heads of one token, so that the rotation's angles are loaded once for them.  (The norms' weights are loaded for every
// head, from L1: the 64 registers a thread that four CTAs an SM leave have no room for them and spill 12 to 16 bytes as it is.)
// The decisions of the quantiser follow the vector's values, so each operation is rounded on its
// own: the result is that of the formulas in fp32 whatever the layout.  Bound by instructions (the norm's two
// sums, the rotation and the quotients of the codes; 73 % of the issue slots) at some twice to three times what its bytes need (2 in per
// value, 2 or 9/16 out): 8192 tokens of 24 + 2 * 4 heads of 256, norms and a rotation of 64: 77 us.
template <int D>
__global__ void __launch_bounds__(kAppendThreads, 4) k_kv_append(const AppendLaunch p, const int steps, const int units) {
  constexpr int LANES = D / 8, HEADS = 32 / LANES;
  const int lane = threadIdx.x & 31, sub = lane % LANES, d = sub * 8;
  const int per_token = p.q_heads + 2 * p.cache.heads;
  const int64_t unit = blockIdx.x * (int64_t)(kAppendThreads / 32) + (threadIdx.x >> 5);
  if (unit >= p.T * units) return;
  const int64_t t = unit >> 32 ? unit / units : (uint32_t)unit / (uint32_t)units;
  int h = (int)(unit - t * units) * steps * HEADS + lane / LANES;
  const __nv_bfloat16* q = reinterpret_cast<const __nv_bfloat16*>(p.q) + t * p.ldq + d;
  const __nv_bfloat16* k = reinterpret_cast<const __nv_bfloat16*>(p.k) + t * p.ldk + d;
  const __nv_bfloat16* v = reinterpret_cast<const __nv_bfloat16*>(p.v) + t * p.ldv + d;
  const int64_t slot = p.slots[t];
  const bool kept = slot >= 0 && slot < p.cache.slots;
  const int in = kept ? (int)(slot & (p.cache.page_size - 1)) : 0, r = in % kKvTile;
  uint8_t* const tile0 = kv_tile<D>(p.cache, kept ? slot >> p.cache.page_shift : 0, 0, in);

  // the rotation of this lane's columns
  const int half = p.rot >> 1;
  const bool inside = d < p.rot, low = d < half;
  bool known = true;
  int from = lane;        // the lane that holds the other of each pair
  float c[8], sn[8];
  if (p.rot) {
    const int pos = p.positions[t];
    known = pos >= 0 && pos < p.table_rows;
    if (inside) {
      const float* row = p.table + (known ? (int64_t)pos * p.rot : 0);
      if (p.interleaved) {
        const float4 c4 = *reinterpret_cast<const float4*>(row + (d >> 1));
        const float4 s4 = *reinterpret_cast<const float4*>(row + half + (d >> 1));
        c[0] = c4.x, c[1] = c4.y, c[2] = c4.z, c[3] = c4.w;
        sn[0] = s4.x, sn[1] = s4.y, sn[2] = s4.z, sn[3] = s4.w;
      } else {
        // half / 8 lanes away (rot is a multiple of 16)
        from = low ? lane + half / 8 : lane - half / 8;
        const int at = low ? d : d - half;
        const float4* cp = reinterpret_cast<const float4*>(row + at);
        const float4* sp = reinterpret_cast<const float4*>(row + half + at);
        const float4 c0 = cp[0], c1 = cp[1], s0 = sp[0], s1 = sp[1];
        c[0] = c0.x, c[1] = c0.y, c[2] = c0.z, c[3] = c0.w, c[4] = c1.x, c[5] = c1.y, c[6] = c1.z, c[7] = c1.w;
        // of a cos - b sin the second has a minus sign, of b cos + a sin a plus
        const uint32_t sign = low ? 0x80000000u : 0u;
        const float s8[8] = {s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) sn[i] = __uint_as_float(__float_as_uint(s8[i]) ^ sign);
      }
    }
  }

  auto fetch = [&](int at) {
    const int hh = min(at, per_token - 1), kv = hh - p.q_heads;
    const __nv_bfloat16* src = kv < 0 ? q + (int64_t)hh * D : kv < p.cache.heads ? k + (int64_t)kv * D : v + (int64_t)(kv - p.cache.heads) * D;
    return *reinterpret_cast<const uint4*>(src);
  };
  uint4 next = fetch(h);
#pragma unroll 1
  for (int s = 0; s < steps; ++s, h += HEADS) {
    // every lane stays for the shuffles; one past the last head repeats it and stores nothing
    const bool live = h < per_token;
    const int hh = live ? h : per_token - 1;
    const bool is_q = hh < p.q_heads, is_k = !is_q && hh < p.q_heads + p.cache.heads;
    const int kvh = hh - p.q_heads - (is_k ? 0 : p.cache.heads);
    const uint4 raw = next;
    if (s + 1 < steps) next = fetch(h + HEADS);
    float x[8];
    unpack8(raw, x);
    const bool turned = is_q || is_k;
    if (__any_sync(0xffffffffu, turned)) {
      if (p.k_norm) {
        uint32_t mag = magnitude8(raw);
        if constexpr (LANES == 32) {
          mag = __reduce_max_sync(0xffffffffu, mag);
        } else {
#pragma unroll
          for (int m = 1; m < LANES; m <<= 1) mag = max(mag, __shfl_xor_sync(0xffffffffu, mag, m));
        }
        const float ms = __fmul_rn(sum_squares<LANES>(x, mag), 1.0f / D);
        const float inv = __frcp_rn(__fsqrt_rn(__fadd_rn(ms, p.eps)));
        if (turned) {
          float w[8];
          load_norm8(is_q ? p.q_norm : p.k_norm, p.norms_fp32, d, w);
#pragma unroll
          for (int i = 0; i < 8; i += 2)
            split(mul2(mul2(pair(x[i], x[i + 1]), pair(inv, inv)), pair(w[i], w[i + 1])), x[i], x[i + 1]);
        }
      }
      if (p.rot) {
        if (p.interleaved) {
          if (inside && turned) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float a = x[2 * i], b = x[2 * i + 1];
              x[2 * i] = __fsub_rn(__fmul_rn(a, c[i]), __fmul_rn(b, sn[i]));
              x[2 * i + 1] = __fadd_rn(__fmul_rn(b, c[i]), __fmul_rn(a, sn[i]));
            }
          }
        } else {
          float o[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) o[i] = __shfl_sync(0xffffffffu, x[i], from);
          if (inside && turned) {
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = __fadd_rn(__fmul_rn(x[i], c[i]), __fmul_rn(o[i], sn[i]));
          }
        }
        if (inside && turned && !known) {
#pragma unroll
          for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(0x7FC00000u);
        }
      }
    }
    if (is_q && live)
      *reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(p.q_out) + t * p.ldo + (int64_t)hh * D + d) = pack8(x);
    if (!__any_sync(0xffffffffu, !is_q)) continue;

    // a scale group is two lanes; an inf or NaN in it shows in its exponent bits
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(x[i]) & 0x7FFFFFFFu);
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    if (is_q || !live || !kept) continue;
    const float g = (is_k ? p.cache.k_scale : p.cache.v_scale)[kvh];
    const bool bad = top >= 0x7F800000u;
    const AqNvGroup a = aq_nv_group(bad ? 0.0f : __uint_as_float(top), g, __fmul_rn(6.0f, g));
    const uint32_t codes = bad || a.step == 0.0f ? 0u : quotient_codes(x, a.d);
    uint8_t* tile = tile0 + (int64_t)kvh * (p.cache.page_size / kKvTile) * kv_tile_bytes(D);
    *reinterpret_cast<uint32_t*>(tile + (is_k ? kv_k_code(D, r, d / 2) : kv_v_code(D, r, d / 2))) = codes;
    if ((sub & 1) == 0)
      tile[is_k ? kv_k_scale(D, r, d / 16) : kv_v_scale(D, r, d / 16)] = (uint8_t)(bad ? 0x7Fu : a.sbyte);
  }
}

// One thread per (token, head, 16 values): their 8 code bytes and scale byte of K and of V.
template <int D, int DIR>  // 0 put, 1 get
__global__ void __launch_bounds__(256) k_kv_move(const KvMoveLaunch p) {
  constexpr int GROUPS = D / 16;
  const int64_t i = blockIdx.x * (int64_t)256 + threadIdx.x;
  if (i >= p.T * p.cache.heads * GROUPS) return;
  const int g = (int)(i % GROUPS);
  const int64_t th = i / GROUPS, t = th / p.cache.heads;
  const int h = (int)(th - t * p.cache.heads);
  const int64_t slot = p.slots[t];
  const bool there = slot >= 0 && slot < p.cache.slots;
  const int in = there ? (int)(slot & (p.cache.page_size - 1)) : 0, r = in % kKvTile;
  uint8_t* tile = kv_tile<D>(p.cache, there ? slot >> p.cache.page_shift : 0, h, in);
  const int code_at[2] = {kv_k_code(D, r, g * 8), kv_v_code(D, r, g * 8)};
  const int scale_at[2] = {kv_k_scale(D, r, g), kv_v_scale(D, r, g)};
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    uint2* codes = reinterpret_cast<uint2*>(tile + code_at[w]);
    if constexpr (DIR == 0) {
      if (there) {
        *codes = reinterpret_cast<const uint2*>(w ? p.v_codes : p.k_codes)[i];
        tile[scale_at[w]] = (w ? p.v_scales : p.k_scales)[i];
      }
    } else {
      const uint2 c = there ? *codes : make_uint2(0, 0);
      const uint32_t sb = there ? tile[scale_at[w]] : 0;
      reinterpret_cast<uint2*>(w ? p.v_codes : p.k_codes)[i] = c;
      (w ? p.v_scales : p.k_scales)[i] = (uint8_t)sb;
    }
  }
}

// One thread per (token, head, 8 values), of K and of V: a warp's stores are whole lines.  Bound by
// the latency of slot, codes and store; 8192 tokens of 4 heads of 256: 10.6 us (13.4 with 16 values a thread).
template <int D>
__global__ void __launch_bounds__(256) k_kv_read(const KvMoveLaunch p) {
  constexpr int PARTS = D / 8;
  const int64_t i = blockIdx.x * (int64_t)256 + threadIdx.x;
  if (i >= p.T * p.cache.heads * PARTS) return;
  const int part = (int)(i % PARTS);
  const int64_t th = i / PARTS, t = th >> 32 ? th / p.cache.heads : (uint32_t)th / (uint32_t)p.cache.heads;
  const int h = (int)(th - t * p.cache.heads);
  const int64_t slot = p.slots[t];
  const bool there = slot >= 0 && slot < p.cache.slots;
  const int in = there ? (int)(slot & (p.cache.page_size - 1)) : 0, r = in % kKvTile;
  const uint8_t* tile = kv_tile<D>(p.cache, there ? slot >> p.cache.page_shift : 0, h, in);
  const int code_at[2] = {kv_k_code(D, r, part * 4), kv_v_code(D, r, part * 4)};
  const int scale_at[2] = {kv_k_scale(D, r, part >> 1), kv_v_scale(D, r, part >> 1)};
  uint32_t codes[2], sb[2];
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    codes[w] = there ? *reinterpret_cast<const uint32_t*>(tile + code_at[w]) : 0;
    sb[w] = there ? tile[scale_at[w]] : 0;
  }
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    const float global = (w ? p.cache.v_scale : p.cache.k_scale)[h];
    const float step = __half2float(__ushort_as_half((unsigned short)e4m3x2_to_f16x2(sb[w])));
    uint32_t f[4];
    e2m1x8_to_f16x8(codes[w], f[0], f[1], f[2], f[3]);
    float x[8];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const float2 v = __half22float2(bits_h2(f[q]));
      x[2 * q] = there ? v.x * step * global : 0.0f;
      x[2 * q + 1] = there ? v.y * step * global : 0.0f;
    }
    reinterpret_cast<uint4*>(w ? p.v : p.k)[i] = pack8(x);
  }
}

template <int D>
cudaError_t move(const KvMoveLaunch& L, int dir, cudaStream_t s) {
  const int64_t items = L.T * L.cache.heads * (dir == 2 ? D / 8 : D / 16);
  const unsigned blocks = (unsigned)((items + 255) / 256);
  if (dir == 0) k_kv_move<D, 0><<<blocks, 256, 0, s>>>(L);
  else if (dir == 1) k_kv_move<D, 1><<<blocks, 256, 0, s>>>(L);
  else k_kv_read<D><<<blocks, 256, 0, s>>>(L);
  return cudaGetLastError();
}

template <int D>
cudaError_t append(const AppendLaunch& L, cudaStream_t s) {
  constexpr int kHeads = 32 / (D / 8), kWarps = kAppendThreads / 32;
  const int64_t all = (L.q_heads + 2 * L.cache.heads + kHeads - 1) / kHeads;
  // a few thousand warps fill the GPU; beyond them a warp takes up to 32 steps of its token (8192 tokens of 32 heads of 256, read
  // back: 129 us with 2 steps, 92 with 8, 86.5 with 16, 84.7 with 32)
  const int64_t fill = L.T * all / 8192;
  int64_t steps = fill < 1 ? 1 : fill > 32 ? 32 : fill, units = (all + steps - 1) / steps;
  if (L.T * units / kWarps > (int64_t)1 << 30) steps = all, units = 1;  // more blocks than a grid has
  k_kv_append<D><<<(unsigned)((L.T * units + kWarps - 1) / kWarps), kAppendThreads, 0, s>>>(L, (int)steps, (int)units);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_append(const AppendLaunch& L, int head_dim, cudaStream_t s) {
  return head_dim == 64 ? append<64>(L, s) : head_dim == 128 ? append<128>(L, s) : append<256>(L, s);
}

cudaError_t launch_kv_move(const KvMoveLaunch& L, int head_dim, int dir, cudaStream_t s) {
  return head_dim == 64 ? move<64>(L, dir, s) : head_dim == 128 ? move<128>(L, dir, s) : move<256>(L, dir, s);
}

}  // namespace vt
