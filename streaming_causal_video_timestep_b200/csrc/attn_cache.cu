// la_op_attention_cache_fp8 for few query rows of a key head (single tokens, short
// drafts), and the join of the pieces of a split key axis.
//
// k_attn_cache_rows: one CTA takes 16 rows (query token x head of the key head's
// group) and one piece of the keys; its 4 warps take 16 keys at a time in turn, each
// with a running maximum and sum of its own, joined in shared memory at the end.
// Bound: HBM, every K and V code read once (for up to 16 rows).  A warp keeps
// STAGES - 1 steps of 16 keys (4 KB at D = 128) under way with cp.async into a ring
// of its own, so no warp waits for another; 16-byte chunks are placed by chunk ^ row
// so that the reads below meet no bank twice at D = 128.
//
// The products run on mma.sync m16n8k16 (fp16 operands, fp32 sums): at 16 rows the
// tensor work is a quarter of what HBM allows, and the operands need no shared
// memory, because a contraction may visit its index in any order:
//   S = Q K^T: lane c = lane % 4 of a key's group holds bytes 16c .. 16c+15 (and
//     64 + 16c ..) of the key's row, so the k index of the MMA step that uses bytes
//     4i .. 4i+3 of them stands for head dims 16c + 4i + {0, 1 | 2, 3}; Q is laid out
//     the same way once.
//   O = P V: the MMA's n index lane / 4 stands for head dims (D/8) * n + jn of its
//     jn-th tile, so a lane reads (D/8) consecutive bytes of the 4 keys whose P it
//     holds.
//   The n-th score column of an 8-key group stands for key n ^ 4 (n & 1) of it, which
//     spreads the rows that one quarter warp reads over the swizzle in both products.
// e4m3 codes are exact in fp16; q is scaled to fp16 by a power of two per row.  The
// key page's scale multiplies the scores; the value page's scale enters P's exponent
// (and leaves the normaliser again), so P V needs no multiplications of its own.  Where
// scales lie so far apart that P flushes to 0, the normaliser does without them (see
// LA_CACHE_SPREAD).
#include "attn_cache.cuh"

namespace {

constexpr int WARPS = 4;
constexpr int STAGES = 4;

__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void cp_async16(void* dst, const void* src, bool on) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(on ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async4(void* dst, const void* src, bool on) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(on ? 4 : 0) : "memory");
}

// One step's 16 keys in shared memory: codes as [16][D], chunk ch of row r at slot
// ch ^ (r & 7) (D = 128) or ch ^ (r / 2 & 3) (D = 64), and the page's scales.
template <int D> struct Step {
  uint8_t k[16 * D], v[16 * D];
};
template <int D> __device__ __forceinline__ int slot_of(int r, int ch) { return r * D + ((ch ^ (D == 128 ? r & 7 : r >> 1 & 3)) << 4); }

template <int D> constexpr size_t rows_smem() {
  const size_t ring = WARPS * STAGES * sizeof(Step<D>), join = WARPS * 16 * D * 4;
  return ring > join ? ring : join;
}

// HALVES: 8-row halves of the MMA's 16 rows that hold rows of this call; an empty half
// costs its part of the softmax otherwise (at 1 row, 16 x 40 heads over up to 14040 keys:
// 261 us, 273 with both).
template <typename T, int D, int HALVES>
__global__ void __launch_bounds__(WARPS * 32, 3)
k_attn_cache_rows(const __grid_constant__ AttnCacheParams p) {
  if (p.nsplit > 1) launch_dependents();    // the join may take its place; it waits for this grid's end
  const int b = blockIdx.z, hk = blockIdx.y;
  const int split = blockIdx.x % p.nsplit, tile = blockIdx.x / p.nsplit;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, n = lane >> 2, c = lane & 3;
  // Pieces are of the same length for every sequence, set by the call's bound of the
  // keys (the last takes what is left), so the first table entries are read beside the
  // sequence's lengths.
  const int s0 = split * p.piece_steps;
  int early[STAGES];
#pragma unroll
  for (int i = 0; i < STAGES; ++i) {
    const int at = (s0 + warp + i * WARPS) * 16 >> p.page_shift;
    early[i] = at < p.max_pages ? __ldg(p.block_table + static_cast<long long>(b) * p.max_pages + at) : -1;
  }
  const CacheSeq s = cache_seq(p, b);
  if (s.bad && blockIdx.x == 0 && hk == 0 && threadIdx.x == 0) raise_device_error(p.err, LA_DEVERR_BAD_DESC);
  const int G = p.heads / p.kv_heads;
  const int rows = s.n * G, r0 = tile * 16;
  if (r0 >= rows) return;

  const int last = min(rows, r0 + 16) - 1;
  const int keys = cache_limit(p, s, last / G);                 // limits do not fall along the rows
  const int steps = (keys + 15) / 16;
  const int low = cache_limit(p, s, r0 / G);                    // and the tile's first row has the least
  const int s1 = split == p.nsplit - 1 ? steps : min(steps, s0 + p.piece_steps);

  // The first steps' copies are under way while Q is brought in.
  extern __shared__ __align__(16) uint8_t ring_raw[];
  __shared__ float2 scales[WARPS][STAGES];
  Step<D>* ring = reinterpret_cast<Step<D>*>(ring_raw) + warp * STAGES;
  // Page of step st (-1: behind the end, or none): looked up one step before its copies start.
  auto page_of = [&](int st) { return st < s1 ? cache_page(p, b, st * 16) : -1; };
  auto fetch = [&](int st, int pg, int slot) {
    if (st < s1) {
      const bool on = pg >= 0;
      const long long plane = static_cast<long long>(on ? pg : 0) * p.kv_heads + hk;
      const long long at = plane * (p.page_tokens * D) + (st * 16 & (p.page_tokens - 1)) * D;
      const int valid = on ? keys - st * 16 : 0;             // rows behind the last key become zeros
      Step<D>& x = ring[slot];
      const uint8_t* kp = p.k_pages + at + lane * 16;
      const uint8_t* vp = p.v_pages + at + lane * 16;
      if (valid >= 16) {
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
          const int q = i * 32 + lane, to = slot_of<D>(q / (D / 16), q % (D / 16));
          cp_async16(x.k + to, kp + i * 512);
          cp_async16(x.v + to, vp + i * 512);
        }
      } else {
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
          const int q = i * 32 + lane, r = q / (D / 16), to = slot_of<D>(r, q % (D / 16));
          cp_async16(x.k + to, kp + i * 512, r < valid);
          cp_async16(x.v + to, vp + i * 512, r < valid);
        }
      }
      if (lane < 2) cp_async4(lane ? &scales[warp][slot].y : &scales[warp][slot].x, (lane ? p.v_scale : p.k_scale) + plane, on);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");     // one group a step, empty ones too
  };
  int st = s0 + warp, pg = st < s1 ? cache_page_checked(p, early[0]) : -1;
#pragma unroll
  for (int i = 0; i < STAGES - 1; ++i) {
    const int nx = st + (i + 1) * WARPS < s1 ? cache_page_checked(p, early[i + 1]) : -1;
    fetch(st + i * WARPS, pg, i);
    pg = nx;
  }

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
    for (int j = 0; j < D / 64; ++j) {
      if (p.q_vec) {
        uint4 u[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
        if (on) {
          u[0] = __ldg(reinterpret_cast<const uint4*>(q + j * 64 + c * 16));
          u[1] = __ldg(reinterpret_cast<const uint4*>(q + j * 64 + c * 16) + 1);
        }
#pragma unroll
        for (int e = 0; e < 16; ++e) f[j][e] = q_to_f32(reinterpret_cast<const T*>(u)[e]);
      } else {
#pragma unroll
        for (int e = 0; e < 16; ++e) f[j][e] = on ? q_to_f32(q[j * 64 + c * 16 + e]) : 0.f;
      }
#pragma unroll
      for (int e = 0; e < 16; ++e) amax = max(amax, __float_as_uint(f[j][e]) & 0x7fffffffu);
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
  float o[D / 8][4];
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f}, top_lv = -INFINITY;
#pragma unroll
  for (int i = 0; i < D / 8; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) o[i][e] = 0.f;

  for (int slot = 0; st < s1; st += WARPS, slot = (slot + 1) % STAGES) {
    const int ahead = st + (STAGES - 1) * WARPS;
    const int nx = page_of(ahead + WARPS);
    asm volatile("cp.async.wait_group %0;" ::"n"(STAGES - 2) : "memory");
    __syncwarp();                                            // every lane's copies of this step, and its reads of the last one
    fetch(ahead, pg, (slot + STAGES - 1) % STAGES);
    pg = nx;
    const Step<D>& cur = ring[slot];
    const float ks = scales[warp][slot].x, vs = scales[warp][slot].y;
    float x[2][4];
#pragma unroll
    for (int nt = 0; nt < 2; ++nt) {
      x[nt][0] = x[nt][1] = x[nt][2] = x[nt][3] = 0.f;
#pragma unroll
      for (int j = 0; j < D / 64; ++j) {
        const uint4 u = *reinterpret_cast<const uint4*>(cur.k + slot_of<D>(nt * 8 + (n ^ (n & 1) << 2), 4 * j + c));
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int e = 0; e < 4; ++e)
          mma16816(x[nt], qa[j * 4 + e], e4m3x2_f16x2_lo(w[e]), e4m3x2_f16x2_hi(w[e]));
      }
    }
    // x[nt][2 i + e]: row n + 8 i, key 8 nt + ((2 c + e) ^ 4 e)
    const float lv = __log2f(vs);
    float rv = __frcp_rn(vs);
    const bool far = lv < top_lv - LA_CACHE_SPREAD;          // of all the steps before
    top_lv = fmaxf(top_lv, lv);
    float mt[HALVES];
    const bool full = st * 16 + 16 <= low;                   // no row of the tile is masked here
#pragma unroll
    for (int i = 0; i < HALVES; ++i) {
      const float a = sc[i] * ks;
#pragma unroll
      for (int nt = 0; nt < 2; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) x[nt][2 * i + e] = fmaf(x[nt][2 * i + e], a, lv);
      if (!full) {
#pragma unroll
        for (int nt = 0; nt < 2; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            if (st * 16 + nt * 8 + ((2 * c + e) ^ e << 2) >= lim[i]) x[nt][2 * i + e] = -INFINITY;
      }
      mt[i] = fmaxf(fmaxf(x[0][2 * i], x[0][2 * i + 1]), fmaxf(x[1][2 * i], x[1][2 * i + 1]));
    }
    bool need = mt[0] > m[0] + LA_CACHE_P_TAU;
    if (HALVES == 2) need = need || mt[HALVES - 1] > m[HALVES - 1] + LA_CACHE_P_TAU;
    if (__any_sync(0xffffffffu, need || far)) {
#pragma unroll
      for (int i = 0; i < HALVES; ++i) {
        float t = mt[i];
        t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 1));
        t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 2));
        const float mn = fmaxf(m[i], t);
        const float h = m[i] == mn ? 1.0f : fast_exp2(0.5f * (m[i] - mn)), al = h * h;    // -inf first: 0
        m[i] = mn;
        l[i] = l[i] * h * h;
#pragma unroll
        for (int j = 0; j < D / 8; ++j) {
          o[j][2 * i] *= al;
          o[j][2 * i + 1] *= al;
        }
        if (far) {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float t = x[k >> 1][2 * i + (k & 1)], h = fast_exp2(0.5f * (t - lv + (LA_CACHE_P_BIAS - mn)));
            if (t != -INFINITY) l[i] += h * h;
          }
        }
      }
      if (far) rv = 0.f;                         // counted
    }
    uint32_t pa[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < HALVES; ++i) {
      const float off = LA_CACHE_P_BIAS - (m[i] == -INFINITY ? 0.f : m[i]);
      float e[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) e[k] = fast_exp2(x[k >> 1][2 * i + (k & 1)] + off);
      const float sum = (e[0] + e[1]) + (e[2] + e[3]);
      if (sum != 0.f) l[i] += sum * rv;          // a page that the row does not see adds nothing, whatever its scale
      pa[i] = pack_f16x2(e[0], e[1]);
      pa[2 + i] = pack_f16x2(e[2], e[3]);
    }
    uint32_t vw[4][D / 32];                                           // D/8 bytes of the lane's 4 keys
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = (i >> 1) * 8 + ((2 * c + (i & 1)) ^ (i & 1) << 2);
      if constexpr (D == 128) {
        const uint4 u = *reinterpret_cast<const uint4*>(cur.v + slot_of<D>(r, n));
        vw[i][0] = u.x; vw[i][1] = u.y; vw[i][2] = u.z; vw[i][3] = u.w;
      } else {
        const uint2 u = *reinterpret_cast<const uint2*>(cur.v + slot_of<D>(r, n >> 1) + (n & 1) * 8);
        vw[i][0] = u.x; vw[i][1] = u.y;
      }
    }
#pragma unroll
    for (int w = 0; w < D / 32; ++w) {                                // 4 bytes of each of the 4 keys
      const uint32_t a01 = __byte_perm(vw[0][w], vw[1][w], 0x5140), a23 = __byte_perm(vw[0][w], vw[1][w], 0x7362);
      const uint32_t b01 = __byte_perm(vw[2][w], vw[3][w], 0x5140), b23 = __byte_perm(vw[2][w], vw[3][w], 0x7362);
      mma16816(o[4 * w + 0], pa, e4m3x2_f16x2_lo(a01), e4m3x2_f16x2_lo(b01));
      mma16816(o[4 * w + 1], pa, e4m3x2_f16x2_hi(a01), e4m3x2_f16x2_hi(b01));
      mma16816(o[4 * w + 2], pa, e4m3x2_f16x2_lo(a23), e4m3x2_f16x2_lo(b23));
      mma16816(o[4 * w + 3], pa, e4m3x2_f16x2_hi(a23), e4m3x2_f16x2_hi(b23));
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");

  // Join the warps: o[j][2 i + e] is row n + 8 i, head dim (D/8) (2 c + e) + j.
  __shared__ float sm[WARPS][16], sl[WARPS][16];
  float(*so)[16][D] = reinterpret_cast<float(*)[16][D]>(ring_raw);   // [WARPS][16][D], over the rings
  __syncthreads();                                                    // no warp reads its ring any more
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
    l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
    if (c == 0) {
      sm[warp][n + 8 * i] = m[i];
      sl[warp][n + 8 * i] = l[i];
    }
#pragma unroll
    for (int e = 0; e < 2 && r0 + n + 8 * i < rows; ++e)
#pragma unroll
      for (int j = 0; j < D / 8; ++j) so[warp][n + 8 * i][(D / 8) * (2 * c + e) + j] = o[j][2 * i + e];
  }
  __syncthreads();
  for (int q = threadIdx.x; q < min(16, rows - r0) * (D / 4); q += WARPS * 32) {
    const int r = q / (D / 4), d4 = q % (D / 4) * 4;
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) M = fmaxf(M, sm[w][r]);
    float L = 0.f, a[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
      const float h = sm[w][r] == M ? 1.0f : fast_exp2(0.5f * (sm[w][r] - M)), f = h * h;
      L += sl[w][r] * h * h;
#pragma unroll
      for (int e = 0; e < 4; ++e) a[e] += so[w][r][d4 + e] * f;
    }
    const int tok = s.q0 + (r0 + r) / G, head = hk * G + (r0 + r) % G;
    if (p.nsplit > 1) {
      const long long row = (static_cast<long long>(split) * p.batch + b) * p.max_q * p.heads + (r0 + r) / G * p.heads + head;
      *reinterpret_cast<float4*>(p.part_o + row * D + d4) = make_float4(a[0], a[1], a[2], a[3]);
      if (d4 == 0) p.part_ml[row] = make_float2(M, L);
    } else {
      cache_store4<T>(p, tok, head, d4, a, L);
    }
  }
}

// Joins the pieces of (token, head) rows: o = sum o_s 2^(m_s - M) / sum l_s 2^(m_s - M).
// `wpr` warps of a CTA share a row, each with its pieces' own maximum, and the first of
// them joins what they found.  A lane holds 4 head dims; it reads the (maximum,
// normaliser) of one piece of each 32, so the sums' loads wait for nothing (222 pieces
// of 16 rows: 30 us with the pieces, 37 when a warp read them one after the other).
constexpr int JOIN_WARPS = 8, JOIN_MAX_WARPS = 32;

template <typename T, int D, bool FEW>
__global__ void __launch_bounds__(JOIN_MAX_WARPS * 32)
k_attn_cache_join(const __grid_constant__ AttnCacheParams p, int wpr) {
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, part = warp % wpr;
  const long long row = blockIdx.x * static_cast<long long>(blockDim.x / 32 / wpr) + warp / wpr;
  const long long all = FEW ? static_cast<long long>(p.batch) * p.max_q * p.heads : (p.units - p.full) * 256LL;
  const long long at = min(row, all - 1);
  const int G = p.heads / p.kv_heads;
  int b, head;
  long long q;                                    // query of the sequence
  if constexpr (FEW) {
    b = static_cast<int>(at / (p.max_q * p.heads));
    head = static_cast<int>(at % p.heads);
    q = at / p.heads % p.max_q;
  } else {
    const CacheUnit u = cache_unit(p, p.full + static_cast<int>(at / 256));
    const long long rr = u.pair * 256LL + at % 256;
    b = u.b;
    head = u.hk * G + static_cast<int>(rr % G);
    q = rr / G;
  }
  const CacheSeq s = cache_seq(p, b);
  const bool on = row < all && q < s.n;           // rows of no sequence stay as they are
  const long long tok = s.q0 + q;
  grid_dependency_wait();
  float M = -INFINITY, L = 0.f, a[4] = {0.f, 0.f, 0.f, 0.f};
  const int d4 = lane * 4;
  if (on) {
    const float2* ml = p.part_ml + row;
    const float* po = p.part_o + row * D + d4;
    const long long step = all * wpr;
    for (int i = part + lane * wpr; i < p.nsplit; i += 32 * wpr) M = fmaxf(M, ml[i * all].x);
#pragma unroll
    for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    for (int i0 = part; i0 < p.nsplit; i0 += 32 * wpr) {
      const int mine = i0 + lane * wpr;
      float2 w = make_float2(-INFINITY, 0.f);
      if (mine < p.nsplit) w = ml[mine * all];
      const float h = w.x == M ? 1.0f : fast_exp2(0.5f * (w.x - M)), f = h * h;
      if (mine < p.nsplit) L += w.y * h * h;
      const int n = min(32, (p.nsplit - i0 + wpr - 1) / wpr);
#pragma unroll 8
      for (int k = 0; k < n; ++k) {
        const float g = __shfl_sync(0xffffffffu, f, k);
        if (d4 < D) {
          const float4 v = *reinterpret_cast<const float4*>(po + (i0 * all + k * step) * D);
          a[0] += v.x * g; a[1] += v.y * g; a[2] += v.z * g; a[3] += v.w * g;
        }
      }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
  }
  if (wpr > 1) {
    __shared__ float sm[JOIN_MAX_WARPS], sl[JOIN_MAX_WARPS];
    __shared__ float4 so[JOIN_MAX_WARPS][32];
    if (lane == 0) {
      sm[warp] = M;
      sl[warp] = L;
    }
    so[warp][lane] = make_float4(a[0], a[1], a[2], a[3]);
    __syncthreads();
    if (part != 0) return;
    float X = M;
    for (int w = 1; w < wpr; ++w) X = fmaxf(X, sm[warp + w]);
    L = 0.f;
    a[0] = a[1] = a[2] = a[3] = 0.f;
    for (int w = 0; w < wpr; ++w) {
      const float h = sm[warp + w] == X ? 1.0f : fast_exp2(0.5f * (sm[warp + w] - X)), f = h * h;
      const float4 v = so[warp + w][lane];
      L += sl[warp + w] * h * h;
      a[0] += v.x * f; a[1] += v.y * f; a[2] += v.z * f; a[3] += v.w * f;
    }
  }
  if (on && d4 < D) cache_store4<T>(p, tok, head, d4, a, L);
}

template <typename T, int D>
cudaError_t launch_rows(const AttnCacheParams& p, cudaStream_t st) {
  const long long rows = static_cast<long long>(p.max_q) * (p.heads / p.kv_heads);
  const long long gx = (rows + 15) / 16 * p.nsplit;
  if (gx > 0x7fffffffLL) return cudaErrorInvalidValue;
  auto kern = rows <= 8 ? k_attn_cache_rows<T, D, 1> : k_attn_cache_rows<T, D, 2>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(rows_smem<D>()));
  if (e != cudaSuccess) return e;
  kern<<<dim3(static_cast<unsigned>(gx), p.kv_heads, p.batch), WARPS * 32, rows_smem<D>(), st>>>(p);
  return cudaGetLastError();
}

template <typename T, int D, bool FEW>
cudaError_t launch_join(const AttnCacheParams& p, cudaStream_t st) {
  int wpr = 1;
  while (wpr < JOIN_MAX_WARPS && p.nsplit > 4 * wpr) wpr *= 2;
  const int warps = wpr > JOIN_WARPS ? wpr : JOIN_WARPS;
  const long long rows = FEW ? static_cast<long long>(p.batch) * p.max_q * p.heads : (p.units - p.full) * 256LL;
  const long long ctas = (rows * wpr + warps - 1) / warps;
  if (ctas > 0x7fffffffLL) return cudaErrorInvalidValue;
  // Launched while the pieces still run (they say when); waits for their end on the GPU.
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas));
  cfg.blockDim = dim3(warps * 32);
  cfg.stream = st;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_attn_cache_join<T, D, FEW>, p, wpr);
}

}  // namespace

cudaError_t launch_attn_cache_rows(int dtype, const AttnCacheParams& p, cudaStream_t st) {
  if (dtype == LA_BF16) return p.d == 64 ? launch_rows<__nv_bfloat16, 64>(p, st) : launch_rows<__nv_bfloat16, 128>(p, st);
  return p.d == 64 ? launch_rows<__half, 64>(p, st) : launch_rows<__half, 128>(p, st);
}

template <bool FEW>
static cudaError_t join_by_type(int dtype, const AttnCacheParams& p, cudaStream_t st) {
  if (dtype == LA_BF16)
    return p.d == 64 ? launch_join<__nv_bfloat16, 64, FEW>(p, st) : launch_join<__nv_bfloat16, 128, FEW>(p, st);
  return p.d == 64 ? launch_join<__half, 64, FEW>(p, st) : launch_join<__half, 128, FEW>(p, st);
}

cudaError_t launch_attn_cache_join(int dtype, int few, const AttnCacheParams& p, cudaStream_t st) {
  return few ? join_by_type<true>(dtype, p, st) : join_by_type<false>(dtype, p, st);
}
