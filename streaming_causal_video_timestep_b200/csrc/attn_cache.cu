// la_op_attention_cache_fp8 for few query rows of a key head (single tokens, short
// drafts), and the join of the pieces of a split key axis.
//
// k_attn_cache_rows: one CTA takes 16 rows (query token x head of the key head's
// group) and one piece of the keys; its 4 warps take 16 keys at a time in turn, each
// with a running maximum and sum of its own, joined in shared memory at the end.
// Bound: HBM, every K and V code read once (for up to 16 rows), straight into
// registers in 16-byte loads, the next 16 keys' under way while these are used.
//
// The products run on mma.sync m16n8k16 (fp16 operands, fp32 sums): at 16 rows the
// tensor work is a quarter of what HBM allows, and the operands need no shared
// memory, because a contraction may visit its index in any order:
//   S = Q K^T: lane c = lane % 4 of a key's group holds bytes 16c .. 16c+15 (and
//     64 + 16c ..) of the key's row, so the k index of the MMA step that uses bytes
//     4i .. 4i+3 of them stands for head dims 16c + 4i + {0, 1 | 2, 3}; Q is laid out
//     the same way once.
//   O = P V: the MMA's n index lane / 4 stands for head dims (D/8) * n + jn of its
//     jn-th tile, so a lane reads (D/8) consecutive bytes of its keys 2c, 2c+1, 8+2c,
//     9+2c, which are the keys whose P it holds.
// e4m3 codes are exact in fp16; q is scaled to fp16 by a power of two per row.  The
// key page's scale multiplies the scores; the value page's scale enters P's exponent
// (and leaves the normaliser again), so P V needs no multiplications of its own.
#include "attn_cache.cuh"

namespace {

constexpr int WARPS = 4;

__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// 16 keys' codes of one lane.
template <int D> struct Keys16 {
  uint4 k[2][D / 64];        // key n of 8-key group nt: bytes 16c.. and 64 + 16c..
  uint32_t v[4][D / 32];     // keys 2c, 2c+1, 8+2c, 9+2c: D/8 bytes
  float ks, vs;              // scales of the page
};

template <int D>
__device__ __forceinline__ void load16(const AttnCacheParams& p, int pg, int off, int hk, int valid, int lane, Keys16<D>& x) {
  const int n = lane >> 2, c = lane & 3;
  const long long plane = static_cast<long long>(pg) * p.kv_heads + hk;
  const uint8_t* kp = p.k_pages + plane * (p.page_tokens * D) + static_cast<long long>(off) * D;
  const uint8_t* vp = p.v_pages + plane * (p.page_tokens * D) + static_cast<long long>(off) * D;
  x.ks = __ldg(p.k_scale + plane);
  x.vs = __ldg(p.v_scale + plane);
#pragma unroll
  for (int nt = 0; nt < 2; ++nt)
#pragma unroll
    for (int i = 0; i < D / 64; ++i)
      x.k[nt][i] = __ldg(reinterpret_cast<const uint4*>(kp + (nt * 8 + n) * D + i * 64 + c * 16));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int key = (i >> 1) * 8 + 2 * c + (i & 1);
    if constexpr (D == 128) {
      uint4 w = __ldg(reinterpret_cast<const uint4*>(vp + key * D + n * 16));
      if (key >= valid) w = make_uint4(0, 0, 0, 0);          // behind the last key: codes of any value
      x.v[i][0] = w.x; x.v[i][1] = w.y; x.v[i][2] = w.z; x.v[i][3] = w.w;
    } else {
      uint2 w = __ldg(reinterpret_cast<const uint2*>(vp + key * D + n * 8));
      if (key >= valid) w = make_uint2(0, 0);
      x.v[i][0] = w.x; x.v[i][1] = w.y;
    }
  }
}

template <typename T, int D>
__global__ void __launch_bounds__(WARPS * 32)
k_attn_cache_rows(const __grid_constant__ AttnCacheParams p) {
  const int b = blockIdx.z, hk = blockIdx.y;
  const int split = blockIdx.x % p.nsplit, tile = blockIdx.x / p.nsplit;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, n = lane >> 2, c = lane & 3;
  const CacheSeq s = cache_seq(p, b);
  if (s.bad && blockIdx.x == 0 && hk == 0 && threadIdx.x == 0) raise_device_error(p.err, LA_DEVERR_BAD_DESC);
  const int G = p.heads / p.kv_heads;
  const int rows = s.n * G, r0 = tile * 16;
  if (r0 >= rows) return;

  // Q: rows n and n + 8 of the tile, as MMA operands; sc[]: log2(e)-scaled softmax
  // scale of the row over the power of two that its q carries.
  uint32_t qa[D / 16][4];
  float sc[2];
  int lim[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = r0 + n + 8 * i;
    const bool on = r < rows;
    const T* q = static_cast<const T*>(p.q) + static_cast<long long>(s.q0 + (on ? r / G : 0)) * p.q_st +
                 static_cast<long long>(hk * G + (on ? r % G : 0)) * p.q_sh;
    lim[i] = on ? cache_limit(p, s, r / G) : 0;
    float f[D / 64][16];
    uint32_t amax = 0;
#pragma unroll
    for (int j = 0; j < D / 64; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        f[j][e] = on ? q_to_f32(q[j * 64 + c * 16 + e]) : 0.f;
        amax = max(amax, __float_as_uint(f[j][e]) & 0x7fffffffu);
      }
    amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
    const float g = q_row_scale(amax);
    sc[i] = p.scale_log2 / g;
#pragma unroll
    for (int j = 0; j < D / 64; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        qa[j * 4 + e][i] = pack_f16x2(f[j][4 * e] * g, f[j][4 * e + 1] * g);
        qa[j * 4 + e][2 + i] = pack_f16x2(f[j][4 * e + 2] * g, f[j][4 * e + 3] * g);
      }
  }
  const int last = min(rows, r0 + 16) - 1;
  const int keys = cache_limit(p, s, last / G);                 // limits do not fall along the rows
  const int steps = (keys + 15) / 16;
  const int per = (steps + p.nsplit - 1) / p.nsplit;
  const int s0 = split * per, s1 = min(steps, s0 + per);

  float o[D / 8][4];
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
  for (int i = 0; i < D / 8; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) o[i][e] = 0.f;

  Keys16<D> cur, nxt;
  auto fetch = [&](int st, Keys16<D>& x) {
    const int key0 = st * 16;
    const int pg = cache_page(p, b, key0);
    if (pg >= 0) {
      load16<D>(p, pg, key0 & (p.page_tokens - 1), hk, keys - key0, lane, x);
      return;
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < D / 64; ++j) x.k[i][j] = make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < D / 32; ++j) x.v[i][j] = 0;
    x.ks = x.vs = 1.0f;
  };
  int st = s0 + warp;
  if (st < s1) fetch(st, cur);
  for (; st < s1; st += WARPS) {
    if (st + WARPS < s1) fetch(st + WARPS, nxt);
    float x[2][4];
#pragma unroll
    for (int nt = 0; nt < 2; ++nt) {
      x[nt][0] = x[nt][1] = x[nt][2] = x[nt][3] = 0.f;
#pragma unroll
      for (int j = 0; j < D / 64; ++j) {
        const uint32_t w[4] = {cur.k[nt][j].x, cur.k[nt][j].y, cur.k[nt][j].z, cur.k[nt][j].w};
#pragma unroll
        for (int e = 0; e < 4; ++e)
          mma16816(x[nt], qa[j * 4 + e], e4m3x2_f16x2_lo(w[e]), e4m3x2_f16x2_hi(w[e]));
      }
    }
    // x[nt][2 i + e]: row n + 8 i, key 8 nt + 2 c + e
    const float lv = log2f(cur.vs), rv = 1.0f / cur.vs;
    float mt[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float a = sc[i] * cur.ks;
#pragma unroll
      for (int nt = 0; nt < 2; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int key = st * 16 + nt * 8 + 2 * c + e;
          x[nt][2 * i + e] = key < lim[i] ? fmaf(x[nt][2 * i + e], a, lv) : -INFINITY;
        }
      mt[i] = fmaxf(fmaxf(x[0][2 * i], x[0][2 * i + 1]), fmaxf(x[1][2 * i], x[1][2 * i + 1]));
    }
    if (__any_sync(0xffffffffu, mt[0] > m[0] + LA_CACHE_P_TAU || mt[1] > m[1] + LA_CACHE_P_TAU)) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float t = mt[i];
        t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 1));
        t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 2));
        const float mn = fmaxf(m[i], t);
        const float al = m[i] == mn ? 1.0f : fast_exp2(m[i] - mn);    // -inf first: 0
        m[i] = mn;
        l[i] *= al;
#pragma unroll
        for (int j = 0; j < D / 8; ++j) {
          o[j][2 * i] *= al;
          o[j][2 * i + 1] *= al;
        }
      }
    }
    uint32_t pa[4];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float off = LA_CACHE_P_BIAS - (m[i] == -INFINITY ? 0.f : m[i]);
      float e[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) e[k] = fast_exp2(x[k >> 1][2 * i + (k & 1)] + off);
      const float sum = (e[0] + e[1]) + (e[2] + e[3]);
      if (sum != 0.f) l[i] += sum * rv;          // a page that the row does not see adds nothing, whatever its scale
      pa[i] = pack_f16x2(e[0], e[1]);
      pa[2 + i] = pack_f16x2(e[2], e[3]);
    }
#pragma unroll
    for (int w = 0; w < D / 32; ++w) {                                // 4 bytes of each of the 4 keys
      const uint32_t a01 = __byte_perm(cur.v[0][w], cur.v[1][w], 0x5140), a23 = __byte_perm(cur.v[0][w], cur.v[1][w], 0x7362);
      const uint32_t b01 = __byte_perm(cur.v[2][w], cur.v[3][w], 0x5140), b23 = __byte_perm(cur.v[2][w], cur.v[3][w], 0x7362);
      mma16816(o[4 * w + 0], pa, e4m3x2_f16x2_lo(a01), e4m3x2_f16x2_lo(b01));
      mma16816(o[4 * w + 1], pa, e4m3x2_f16x2_hi(a01), e4m3x2_f16x2_hi(b01));
      mma16816(o[4 * w + 2], pa, e4m3x2_f16x2_lo(a23), e4m3x2_f16x2_lo(b23));
      mma16816(o[4 * w + 3], pa, e4m3x2_f16x2_hi(a23), e4m3x2_f16x2_hi(b23));
    }
    cur = nxt;
  }

  // Join the warps: o[j][2 i + e] is row n + 8 i, head dim (D/8) (2 c + e) + j.
  __shared__ float sm[WARPS][16], sl[WARPS][16];
  __shared__ float so[WARPS][16][D];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
    l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
    if (c == 0) {
      sm[warp][n + 8 * i] = m[i];
      sl[warp][n + 8 * i] = l[i];
    }
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
      for (int j = 0; j < D / 8; ++j) so[warp][n + 8 * i][(D / 8) * (2 * c + e) + j] = o[j][2 * i + e];
  }
  __syncthreads();
  for (int q = threadIdx.x; q < 16 * (D / 4); q += WARPS * 32) {
    const int r = q / (D / 4), d4 = q % (D / 4) * 4;
    if (r0 + r >= rows) continue;
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) M = fmaxf(M, sm[w][r]);
    float L = 0.f, a[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
      const float f = sm[w][r] == M ? 1.0f : fast_exp2(sm[w][r] - M);
      L += sl[w][r] * f;
#pragma unroll
      for (int e = 0; e < 4; ++e) a[e] += so[w][r][d4 + e] * f;
    }
    const int tok = s.q0 + (r0 + r) / G, head = hk * G + (r0 + r) % G;
    if (p.nsplit > 1) {
      const long long row = (static_cast<long long>(split) * p.tokens + tok) * p.heads + head;
      *reinterpret_cast<float4*>(p.part_o + row * D + d4) = make_float4(a[0], a[1], a[2], a[3]);
      if (d4 == 0) p.part_ml[row] = make_float2(M, L);
    } else {
      cache_store4<T>(p, tok, head, d4, a, L);
    }
  }
}

// One warp joins the pieces of one (token, head) row: o = sum o_s 2^(m_s - M) / sum l_s 2^(m_s - M).
template <typename T, int D>
__global__ void __launch_bounds__(128)
k_attn_cache_join(const __grid_constant__ AttnCacheParams p) {
  const long long row = blockIdx.x * 4LL + threadIdx.x / 32;
  const int lane = threadIdx.x % 32;
  const long long all = static_cast<long long>(p.tokens) * p.heads;
  if (row >= all) return;
  const int tok = static_cast<int>(row / p.heads), head = static_cast<int>(row % p.heads);
  // Rows of no sequence stay as they are.
  int lo = 0, hi = p.batch;
  while (lo < hi) {                               // first b with cu_q[b + 1] > tok
    const int mid = (lo + hi) / 2;
    if (p.cu_q[mid + 1] > tok) hi = mid;
    else lo = mid + 1;
  }
  if (lo == p.batch) return;
  const CacheSeq s = cache_seq(p, lo);
  if (s.bad || tok < s.q0 || tok >= s.q0 + s.n) return;
  float M = -INFINITY;
  for (int i = lane; i < p.nsplit; i += 32) M = fmaxf(M, p.part_ml[i * all + row].x);
#pragma unroll
  for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  float L = 0.f, a[4] = {0.f, 0.f, 0.f, 0.f};
  const int d4 = lane * 4;
  for (int i = 0; i < p.nsplit; ++i) {
    const float2 ml = p.part_ml[i * all + row];
    const float f = ml.x == M ? 1.0f : fast_exp2(ml.x - M);
    L += ml.y * f;
    if (d4 < D) {
      const float4 v = *reinterpret_cast<const float4*>(p.part_o + (i * all + row) * D + d4);
      a[0] += v.x * f; a[1] += v.y * f; a[2] += v.z * f; a[3] += v.w * f;
    }
  }
  if (d4 < D) cache_store4<T>(p, tok, head, d4, a, L);
}

template <typename T, int D>
cudaError_t launch_rows(const AttnCacheParams& p, cudaStream_t st) {
  const long long rows = static_cast<long long>(p.max_q) * (p.heads / p.kv_heads);
  const long long gx = (rows + 15) / 16 * p.nsplit;
  if (gx > 0x7fffffffLL) return cudaErrorInvalidValue;
  k_attn_cache_rows<T, D><<<dim3(static_cast<unsigned>(gx), p.kv_heads, p.batch), WARPS * 32, 0, st>>>(p);
  return cudaGetLastError();
}

template <typename T, int D>
cudaError_t launch_join(const AttnCacheParams& p, cudaStream_t st) {
  const long long all = static_cast<long long>(p.tokens) * p.heads;
  if ((all + 3) / 4 > 0x7fffffffLL) return cudaErrorInvalidValue;
  k_attn_cache_join<T, D><<<ceil_div_i(all, 4), 128, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attn_cache_rows(int dtype, const AttnCacheParams& p, cudaStream_t st) {
  if (dtype == LA_BF16) return p.d == 64 ? launch_rows<__nv_bfloat16, 64>(p, st) : launch_rows<__nv_bfloat16, 128>(p, st);
  return p.d == 64 ? launch_rows<__half, 64>(p, st) : launch_rows<__half, 128>(p, st);
}

cudaError_t launch_attn_cache_join(int dtype, const AttnCacheParams& p, cudaStream_t st) {
  if (dtype == LA_BF16) return p.d == 64 ? launch_join<__nv_bfloat16, 64>(p, st) : launch_join<__nv_bfloat16, 128>(p, st);
  return p.d == 64 ? launch_join<__half, 64>(p, st) : launch_join<__half, 128>(p, st);
}
