// Attention over the paged 8-bit cache: what its two kernels and their combine share.
#pragma once

#include <cuda_fp16.h>

#include "kernels.h"
#include "sm100.cuh"

// P is formed as 2^(t - M + P_BIAS), t the score (log2 domain) plus log2 of the
// value page's scale, M the running maximum of t, raised when t exceeds it by more
// than P_TAU: P <= 2^15 in fp16, and keeps fp16's 11 bits down to 2^-21 of 2^M (2^-31
// in fp16's subnormals).  A raise rescales O; with 4 for P_TAU it came often enough to
// cost 2 % at 4680 x 15600 x 40 x 128.
#define LA_CACHE_P_BIAS 7.0f
#define LA_CACHE_P_TAU 8.0f
// The normaliser counts 2^(s - M + P_BIAS) of every key, s its score alone: a sum of P
// over the page's value scale.  Value scales reach from 2^-64 to 2^120 (the append's),
// so the keys that matter make that a normal fp32 number (M is within P_TAU of a largest
// t, hence at most 2^120 above the largest score), but P on the way to it, or a factor
// between two maxima, may lie below 2^-126 and flush to 0.  Hence:
//   * keys of a page whose value scale lies more than 2^SPREAD below the largest before
//     it are summed without the scale; of the others, 2^-126 / vs at most is flushed,
//     2^(SPREAD - 133) of the normaliser;
//   * sums are taken from one maximum to another by 2^((M - M') / 2), twice.
#define LA_CACHE_SPREAD 90.0f

// Programmatic launch: the next grid of the stream may start, and waits here for the
// end of the grid before it.
__device__ __forceinline__ void launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void grid_dependency_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// One sequence's place in the batch, checked: whatever the device arrays hold,
// rows and keys stay inside the tensors.
struct CacheSeq {
  int q0, n, L;        // first query row, queries, keys
  bool bad;
};
__device__ __forceinline__ CacheSeq cache_seq(const AttnCacheParams& p, int b) {
  CacheSeq s;
  s.q0 = p.cu_q[b];
  const int q1 = p.cu_q[b + 1];
  s.L = p.kv_len[b];
  s.bad = s.q0 < 0 || q1 < s.q0 || q1 > p.tokens || q1 - s.q0 > p.max_q || s.L < 0 ||
          s.L > static_cast<long long>(p.max_pages) * p.page_tokens;
  s.n = s.bad ? 0 : q1 - s.q0;
  if (s.bad) s.L = 0;
  return s;
}
// Keys that query r of the sequence sees: j < limit.
__device__ __forceinline__ int cache_limit(const AttnCacheParams& p, const CacheSeq& s, int r) {
  if (p.causal_block == 0) return s.L;
  const long long lim = static_cast<long long>(s.L) - s.n + (r / p.causal_block + 1LL) * p.causal_block;
  return static_cast<int>(max(0LL, min(lim, static_cast<long long>(s.L))));
}
// Unit of 256 rows: under a causal mask the last rows of a sequence, which have the most
// keys, come first.
struct CacheUnit {
  int b, hk, pair;
};
__device__ __forceinline__ CacheUnit cache_unit(const AttnCacheParams& p, int unit) {
  const int bh = unit / p.pairs;
  return {bh / p.kv_heads, bh % p.kv_heads, p.pairs - 1 - unit % p.pairs};
}
// A page that the table names, -1 (and the error word) if there is no such page.
__device__ __forceinline__ int cache_page_checked(const AttnCacheParams& p, int pg) {
  if (pg >= 0 && pg < p.num_pages) return pg;
  raise_device_error(p.err, LA_DEVERR_BAD_DESC);
  return -1;
}
// Page of the sequence that holds key j (j < L).
__device__ __forceinline__ int cache_page(const AttnCacheParams& p, int b, int j) {
  return cache_page_checked(p, p.block_table[static_cast<long long>(b) * p.max_pages + (j >> p.page_shift)]);
}

// Two e4m3 codes (low 16 bits) to fp16, exactly.
__device__ __forceinline__ uint32_t e4m3x2_f16x2_lo(uint32_t w) {
  uint32_t r;
  asm("{\n\t.reg .b16 l, u;\n\tmov.b32 {l, u}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t}" : "=r"(r) : "r"(w));
  return r;
}
__device__ __forceinline__ uint32_t e4m3x2_f16x2_hi(uint32_t w) {
  uint32_t r;
  asm("{\n\t.reg .b16 l, u;\n\tmov.b32 {l, u}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, u;\n\t}" : "=r"(r) : "r"(w));
  return r;
}

// The power of two that brings a row whose largest |q| has these bits to [2^14, 2^15):
// bf16 (or fp16) times it is exact in fp16 down to 2^-29 of the row's largest.
// 1 for a zero row and one that is not finite.
__device__ __forceinline__ float q_row_scale(uint32_t amax_bits) {
  const int e = static_cast<int>(amax_bits >> 23);
  if (e == 0 || e == 255) return 1.0f;
  return __uint_as_float(static_cast<uint32_t>(min(max(127 + 14 - (e - 127), 1), 254)) << 23);
}

__device__ __forceinline__ float q_to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float q_to_f32(__half v) { return __half2float(v); }

template <typename T> __device__ __forceinline__ uint2 q_pack4(const float (&v)[4]);
template <> __device__ __forceinline__ uint2 q_pack4<__nv_bfloat16>(const float (&v)[4]) {
  return make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
}
template <> __device__ __forceinline__ uint2 q_pack4<__half>(const float (&v)[4]) {
  return make_uint2(pack_f16x2(v[0], v[1]), pack_f16x2(v[2], v[3]));
}
// Four head dims of one output row: a / L, 0 where the row saw no key (L = 0).
template <typename T>
__device__ __forceinline__ void cache_store4(const AttnCacheParams& p, long long tok, int head, int d4, const float (&a)[4], float L) {
  float v[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] = a[e] * (L == 0.f ? 0.f : __frcp_rn(L));
  *reinterpret_cast<uint2*>(static_cast<T*>(p.out) + tok * p.o_st + head * p.o_sh + d4) = q_pack4<T>(v);
  if (p.out32) *reinterpret_cast<float4*>(p.out32 + (tok * p.heads + head) * p.d + d4) = make_float4(v[0], v[1], v[2], v[3]);
}
// Eight of them.
template <typename T>
__device__ __forceinline__ void cache_store8(const AttnCacheParams& p, long long tok, int head, int d8, const float (&a)[8], float L) {
  if (p.o_vec && !p.out32) {
    const float inv = L == 0.f ? 0.f : __frcp_rn(L);
    const float lo[4] = {a[0] * inv, a[1] * inv, a[2] * inv, a[3] * inv}, hi[4] = {a[4] * inv, a[5] * inv, a[6] * inv, a[7] * inv};
    const uint2 x = q_pack4<T>(lo), y = q_pack4<T>(hi);
    *reinterpret_cast<uint4*>(static_cast<T*>(p.out) + tok * p.o_st + head * p.o_sh + d8) = make_uint4(x.x, x.y, y.x, y.y);
    return;
  }
  const float lo[4] = {a[0], a[1], a[2], a[3]}, hi[4] = {a[4], a[5], a[6], a[7]};
  cache_store4<T>(p, tok, head, d8, lo, L);
  cache_store4<T>(p, tok, head, d8 + 4, hi, L);
}
