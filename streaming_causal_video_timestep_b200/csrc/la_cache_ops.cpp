// Op-level C entry points for rotary positions with several axes and the paged
// 8-bit cache: argument checks, the frequency table, the split of the key axis.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "kernels.h"
#include "la_stream.h"

namespace {

int num_sms_current() {
  int dev = 0, sms = 148;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  return sms;
}
int ret(cudaError_t e) { return e == cudaSuccess ? LA_OK : LA_ECUDA; }

constexpr int64_t kMaxRows = 1LL << 30;

bool aligned(const void* p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }
size_t elem_size(int32_t dtype) { return dtype == LA_FP32 ? 4 : 2; }
bool known_dtype(int32_t dtype) { return dtype == LA_BF16 || dtype == LA_FP32 || dtype == LA_FP16; }

// omega_{a,j} = theta^(-j / pairs[a]), as a fraction of a turn in units of 2^-64: one
// exp2l an axis and one multiplication a pair from the last power but at most 8 (long
// double keeps the 64 bits that the product with a position uses; a call on one token
// takes less time than 12 powl).  With up to 15 + 7 factors and the cut to 2^-64 an entry
// is off by 2^-60 turns at most: 2^-60.9 was the most for 1 to 128 pairs and 16 thetas
// from 1 to 1e12, against powers with 113 bits.
bool fill_table(RotaryTable& t, int32_t d, int32_t naxes, const int32_t* pairs, double theta, int32_t half,
                int32_t inverse) {
  t.n = 0;
  t.naxes = naxes;
  t.half = half != 0 && naxes > 0;
  t.inverse = inverse != 0;
  if (naxes < 0 || naxes > LA_MAX_AXES || (naxes > 0 && !pairs)) return false;
  if (naxes > 0 && !(theta >= 1.0 && theta <= 1e12)) return false;
  constexpr long double two_pi = 6.283185307179586476925286766559005768L;
  for (int a = 0; a < naxes; ++a) {
    if (pairs[a] < 0 || pairs[a] > d / 2 - t.n) return false;
    if (pairs[a] == 0) continue;
    const long double step = exp2l(-log2l(theta) / pairs[a]), two = step * step, four = two * two, eight = four * four;
    long double base = 1.0L / two_pi, turns = base;
    for (int j = 0; j < pairs[a]; ++j) {
      if (j > 0 && j % 8 == 0) turns = base *= eight;
      else if (j > 0) turns *= step;
      t.turn[t.n] = static_cast<unsigned long long>(static_cast<long long>(turns * 0x1p64L));   // < 2^62: turns <= 1 / (2 pi)
      t.axis[t.n++] = static_cast<unsigned char>(a);
    }
  }
  return naxes == 0 || t.n > 0;
}

bool strides_fit(int64_t rows, int64_t st, int64_t sh, int32_t heads, int32_t d) {
  return st >= 0 && sh >= 0 && (heads == 1 || sh >= d) && (rows <= 1 || st >= 1) && st <= (1LL << 40) && sh <= (1LL << 40);
}

// An output's rows do not lie over one another: one of the two strides steps over all of the other's.
// (128 bits: a stride may be 2^40, and 2^30 rows or 2^31 heads may lie that far apart.)
bool rows_apart(__int128 rows, __int128 st, __int128 sh, int32_t heads, int32_t d) {
  return rows <= 1 || st >= (heads - 1) * sh + d || (heads == 1 ? st >= d : st >= d && sh >= (rows - 1) * st + d);
}

bool cache_fine(const la_paged_cache* c) {
  if (!c || !c->k_pages || !c->v_pages || !c->k_scale || !c->v_scale || !c->block_table) return false;
  if (!aligned(c->k_pages, 16) || !aligned(c->v_pages, 16) || !aligned(c->k_scale, 4) || !aligned(c->v_scale, 4) ||
      !aligned(c->block_table, 4))
    return false;
  if (c->head_dim != 64 && c->head_dim != 128) return false;
  if (c->page_tokens != 32 && c->page_tokens != 64 && c->page_tokens != 128) return false;
  return c->num_pages >= 1 && c->heads >= 1 && c->heads <= 65535 && c->batch >= 1 && c->batch <= 65535 && c->max_pages >= 1 &&
         static_cast<int64_t>(c->max_pages) * c->page_tokens <= kMaxRows;
}

bool few_rows(int64_t max_q, int32_t heads, int32_t kv_heads) { return max_q * (heads / kv_heads) <= LA_CACHE_FEW_ROWS; }

// How a call is laid out.  Few rows: enough CTAs for 3 on every SM with at least 128
// keys each (one token over 1561 keys x 8 heads: 10.0 us; 11.2 with 256), and pieces of
// about 2048 keys where that makes more, which evens out ragged lengths (16 x 40 heads
// over up to 14040 keys: 262 us; 311 unsplit, 279 with 1024 keys).
// Many rows: one CTA an SM, 256 rows of a (sequence, key head) each.  The units behind
// the last full round of the SMs are split along the keys, into the number of pieces that
// makes the fewest key tiles in a row, a piece counted two tiles longer than it is for
// its start and end and its part of the join (760 units of 122 tiles: 1767 us
// unsplit, 1589 with the last 20 in 7 pieces each).
struct Plan {
  int nsplit = 1, pairs = 0, full = 0, units = 0;
  int64_t part_rows = 0;                           // of all pieces
};
constexpr int kSms = 148;

bool plan_call(Plan& pl, int64_t max_q, int64_t max_kv, int32_t batch, int32_t heads, int32_t kv_heads) {
  if (few_rows(max_q, heads, kv_heads)) {
    const int64_t ctas = static_cast<int64_t>(kv_heads) * batch;
    pl.nsplit = static_cast<int>(std::max({int64_t{1}, std::min((kSms * 3 + ctas - 1) / ctas, max_kv / 128), std::min<int64_t>(max_kv / 2048, 1024)}));
    pl.part_rows = pl.nsplit > 1 ? pl.nsplit * batch * max_q * heads : 0;
    return true;
  }
  const int64_t pairs = (max_q * (heads / kv_heads) + 255) / 256, units = pairs * kv_heads * batch;
  if (units > (1 << 28)) return false;
  const int64_t tail = units % kSms, tiles = (max_kv + 127) / 128;
  int64_t best = INT64_MAX;
  for (int n = 1; n <= 32 && tail > 0 && (n == 1 || tiles / n >= 4); ++n) {
    const int64_t cost = (tail * n + kSms - 1) / kSms * ((tiles + n - 1) / n + 2);
    if (cost < best) best = cost, pl.nsplit = n;
  }
  pl.pairs = static_cast<int>(pairs);
  pl.units = static_cast<int>(units);
  pl.full = static_cast<int>(pl.nsplit > 1 ? units - tail : units);
  pl.part_rows = pl.nsplit > 1 ? pl.nsplit * tail * 256 : 0;
  return true;
}

}  // namespace

extern "C" {

int la_op_rope_axes(int32_t dtype, const void* x, int64_t x_token_stride, int64_t x_head_stride, void* out,
                    int64_t out_token_stride, int64_t out_head_stride, int64_t tokens, int32_t heads, int32_t head_dim,
                    const int32_t* pos, int32_t naxes, const int32_t* pairs, double theta, int32_t half, int32_t inverse,
                    void* cuda_stream) {
  if (!known_dtype(dtype) || tokens < 0 || tokens > kMaxRows || heads < 1 || heads > 65535) return LA_EINVAL;
  if (head_dim < 2 || head_dim > 2 * LA_ROPE_MAX_PAIRS || naxes < 1) return LA_EINVAL;
  if (!strides_fit(tokens, x_token_stride, x_head_stride, heads, head_dim) ||
      !strides_fit(tokens, out_token_stride, out_head_stride, heads, head_dim) ||
      !rows_apart(tokens, out_token_stride, out_head_stride, heads, head_dim))
    return LA_EINVAL;
  RotaryTable tab;
  if (!fill_table(tab, head_dim, naxes, pairs, theta, half, inverse)) return LA_EINVAL;
  if (tokens == 0) return LA_OK;
  if (!x || !out || !pos || !aligned(x, elem_size(dtype)) || !aligned(out, elem_size(dtype)) || !aligned(pos, 4)) return LA_EINVAL;
  RopeAxesParams p{};
  p.x = x;
  p.out = out;
  p.pos = pos;
  p.tokens = tokens;
  p.x_st = x_token_stride;
  p.x_sh = x_head_stride;
  p.o_st = out_token_stride;
  p.o_sh = out_head_stride;
  p.heads = heads;
  p.d = head_dim;
  return ret(launch_rope_axes(dtype, p, tab, num_sms_current(), static_cast<cudaStream_t>(cuda_stream)));
}

int la_op_cache_append_fp8(const la_paged_cache* cache, int32_t dtype, const void* k, int64_t k_token_stride,
                           int64_t k_head_stride, const void* v, int64_t v_token_stride, int64_t v_head_stride,
                           int64_t tokens, const int32_t* cu_new, const int32_t* cache_len, int64_t max_new,
                           const int32_t* pos, int32_t naxes, const int32_t* pairs, double theta, int32_t half,
                           void* cuda_stream) {
  if (!cache_fine(cache) || !known_dtype(dtype) || tokens < 0 || tokens > kMaxRows || max_new < 0 || max_new > kMaxRows)
    return LA_EINVAL;
  if (!strides_fit(tokens, k_token_stride, k_head_stride, cache->heads, cache->head_dim) ||
      !strides_fit(tokens, v_token_stride, v_head_stride, cache->heads, cache->head_dim))
    return LA_EINVAL;
  RotaryTable tab;
  if (!fill_table(tab, cache->head_dim, naxes, pairs, theta, half, 0)) return LA_EINVAL;
  if (!cu_new || !cache_len || (tab.n > 0 && tokens > 0 && !pos) || !aligned(cu_new, 4) || !aligned(cache_len, 4) ||
      !aligned(pos, 4))
    return LA_EINVAL;
  if (tokens == 0 || max_new == 0) return LA_OK;
  if (!k || !v || !aligned(k, elem_size(dtype)) || !aligned(v, elem_size(dtype))) return LA_EINVAL;
  CacheAppendParams p{};
  p.k = k;
  p.v = v;
  p.k_st = k_token_stride;
  p.k_sh = k_head_stride;
  p.v_st = v_token_stride;
  p.v_sh = v_head_stride;
  p.pos = pos;
  p.k_pages = static_cast<uint8_t*>(cache->k_pages);
  p.v_pages = static_cast<uint8_t*>(cache->v_pages);
  p.k_scale = cache->k_scale;
  p.v_scale = cache->v_scale;
  p.block_table = cache->block_table;
  p.cache_len = cache_len;
  p.cu_new = cu_new;
  p.tokens = static_cast<int>(tokens);
  p.batch = cache->batch;
  p.heads = cache->heads;
  p.d = cache->head_dim;
  p.page_tokens = cache->page_tokens;
  p.num_pages = cache->num_pages;
  p.max_pages = cache->max_pages;
  p.max_new = static_cast<int>(std::min(max_new, tokens));
  if (op_error_word(&p.err) != LA_OK) return LA_ECUDA;
  return ret(launch_cache_append(dtype, p, tab, num_sms_current(), static_cast<cudaStream_t>(cuda_stream)));
}

int64_t la_op_attention_cache_fp8_workspace(const la_paged_cache* cache, int64_t tokens, int32_t heads, int64_t max_q,
                                            int64_t max_kv) {
  if (!cache_fine(cache) || heads < 1 || heads % cache->heads != 0 || tokens < 0 || tokens > kMaxRows || max_q < 0 ||
      max_q > kMaxRows || max_kv < 0 || max_kv > kMaxRows)
    return LA_EINVAL;
  Plan pl;
  if (!plan_call(pl, std::min(max_q, tokens), max_kv, cache->batch, heads, cache->heads)) return LA_EINVAL;
  return pl.part_rows * (cache->head_dim * 4LL + 8);
}

int la_op_attention_cache_fp8(const la_paged_cache* cache, int32_t dtype, const void* q, int64_t q_token_stride,
                              int64_t q_head_stride, int64_t tokens, int32_t heads, const int32_t* cu_q,
                              const int32_t* kv_len, int64_t max_q, int64_t max_kv, int32_t causal_block, double scale,
                              void* out, int64_t out_token_stride, int64_t out_head_stride, float* out32, void* workspace,
                              int64_t workspace_bytes, void* cuda_stream) {
  if (!cache_fine(cache) || (dtype != LA_BF16 && dtype != LA_FP16)) return LA_EINVAL;
  if (heads < 1 || heads % cache->heads != 0 || tokens < 0 || tokens > kMaxRows || max_q < 0 || max_q > kMaxRows ||
      max_kv < 0 || max_kv > kMaxRows || causal_block < 0 || !(scale > 0.0 && scale < 1e30))
    return LA_EINVAL;
  if (!strides_fit(tokens, q_token_stride, q_head_stride, heads, cache->head_dim) ||
      !strides_fit(tokens, out_token_stride, out_head_stride, heads, cache->head_dim) ||
      !rows_apart(tokens, out_token_stride, out_head_stride, heads, cache->head_dim))
    return LA_EINVAL;
  if (!cu_q || !kv_len || !aligned(cu_q, 4) || !aligned(kv_len, 4)) return LA_EINVAL;
  const int64_t need = la_op_attention_cache_fp8_workspace(cache, tokens, heads, max_q, max_kv);
  if (need < 0 || workspace_bytes < need || (need > 0 && (!workspace || !aligned(workspace, 16)))) return LA_EINVAL;
  if (tokens == 0 || max_q == 0) return LA_OK;
  if (!q || !out || !aligned(q, 2) || !aligned(out, 8) || out_token_stride % 4 != 0 || out_head_stride % 4 != 0 ||
      !aligned(out32, 16))
    return LA_EINVAL;
  AttnCacheParams p{};
  p.q = q;
  p.out = out;
  p.out32 = out32;
  p.q_vec = aligned(q, 16) && q_token_stride % 8 == 0 && q_head_stride % 8 == 0;
  p.o_vec = aligned(out, 16) && out_token_stride % 8 == 0 && out_head_stride % 8 == 0;
  p.q_st = q_token_stride;
  p.q_sh = q_head_stride;
  p.o_st = out_token_stride;
  p.o_sh = out_head_stride;
  p.k_pages = static_cast<const uint8_t*>(cache->k_pages);
  p.v_pages = static_cast<const uint8_t*>(cache->v_pages);
  p.k_scale = cache->k_scale;
  p.v_scale = cache->v_scale;
  p.block_table = cache->block_table;
  p.kv_len = kv_len;
  p.cu_q = cu_q;
  p.tokens = static_cast<int>(tokens);
  p.batch = cache->batch;
  p.heads = heads;
  p.kv_heads = cache->heads;
  p.d = cache->head_dim;
  p.page_tokens = cache->page_tokens;
  p.page_shift = p.page_tokens == 32 ? 5 : p.page_tokens == 64 ? 6 : 7;
  p.num_pages = cache->num_pages;
  p.max_pages = cache->max_pages;
  p.max_q = static_cast<int>(std::min(max_q, tokens));
  p.causal_block = causal_block;
  p.scale_log2 = static_cast<float>(scale * 1.4426950408889634);
  Plan pl;
  if (!plan_call(pl, p.max_q, max_kv, p.batch, heads, cache->heads)) return LA_EINVAL;
  p.nsplit = pl.nsplit;
  p.piece_steps = static_cast<int>(((max_kv + 15) / 16 + p.nsplit - 1) / p.nsplit);
  p.pairs = pl.pairs;
  p.full = pl.full;
  p.units = pl.units;
  if (p.nsplit > 1) {
    p.part_o = static_cast<float*>(workspace);
    p.part_ml = reinterpret_cast<float2*>(p.part_o + pl.part_rows * p.d);
  }
  if (op_error_word(&p.err) != LA_OK) return LA_ECUDA;
  cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  const bool few = few_rows(p.max_q, heads, cache->heads);
  cudaError_t e = few ? launch_attn_cache_rows(dtype, p, st) : launch_attn_cache_tc(dtype, p, st);
  if (e == cudaSuccess && p.nsplit > 1) e = launch_attn_cache_join(dtype, few, p, st);
  return ret(e);
}

}  // extern "C"
