// la_op_attention_cache_fp8 for many query rows of a key head: tcgen05 (kind::f16),
// two 128-row tiles a CTA.
//
// One CTA = up to 256 rows (query token x head of the key head's group) of one
// sequence and key head, over one piece of the keys in tiles of 128.  16 warps:
//   warp 1       owns tensor memory (512 columns: S_A | S_B | O_A | O_B) and issues
//                the MMAs: PV_A(t), S_A(t+1), PV_B(t), S_B(t+1), ..., so that one
//                tile's softmax runs beside the other's products; warps 0, 2, 3 idle
//   warps 4-11   softmax of tiles A and B, a thread a row; before that they bring Q
//                to shared memory as fp16 under a power of two per row
//   warps 12-15  bring K and V: 16-byte loads of e4m3 codes (page by page, so the
//                page table costs a lookup per 32 keys), one tile ahead in registers,
//                turned into fp16 (exactly) and written to a two-stage ring in the
//                128-byte-swizzled layout that the MMAs read
// The codes are unpacked once for 256 rows; at 64 conversions a clock and SM that
// takes a quarter of the tile's MMA time and runs beside it.  fp16 operands keep q
// and the codes exact and P to 11 bits (e4m3 or bf16 P would not).
//
// Scales: the score of a key is acc * ks * (row factor); log2(vs) enters the
// exponent, so a page's P carries its value scale and the normaliser takes it out
// again (sum * 1 / vs): scales cost no instruction an element beyond the scale and
// offset that the exponent needs anyway.
#include <cstdio>

#include "attn_cache.cuh"

namespace {

constexpr int THREADS = 512;
constexpr int LAUNCH_REGS = 128;            // 65536 / 512
constexpr int REGS_LOW = 40;                // warps 0-3
constexpr int REGS_LOAD = 104;              // warps 12-15
constexpr int REGS_SOFT = 184;              // warps 4-11
static_assert(128 * (REGS_LOW + REGS_LOAD + 2 * REGS_SOFT) <= THREADS * LAUNCH_REGS, "register split exceeds the launch");
constexpr uint32_t BOX = 16384;             // 128 rows x 64 fp16, 128-byte swizzle
constexpr uint32_t TMEM_COLS = 512;
constexpr int NSC = 8;                      // ring of the tiles' scales, longer than any K ring
static_assert(NSC > 4, "the scales' ring must outlast the K ring");

template <int D> __host__ __device__ constexpr uint32_t tile_bytes() { return D / 64 * BOX; }
template <int D> __host__ __device__ constexpr int stages() { return D == 64 ? 4 : 2; }
template <int D> __host__ __device__ constexpr size_t smem_bytes() {
  return 1024 + 2 * tile_bytes<D>() + stages<D>() * 2 * tile_bytes<D>() + NSC * 64 + 512;
}

template <int N>
__device__ __forceinline__ void regs_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void regs_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }

__device__ __forceinline__ uint32_t s_col(int w) { return static_cast<uint32_t>(w * 128); }
__device__ __forceinline__ uint32_t o_col(int w) { return static_cast<uint32_t>(256 + w * 128); }

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// One row's scores of a key tile (raw accumulators in s) to P (fp16 pairs) and the
// row's share of the normaliser.  sc[c]: the 32-key chunk's (ks, log2 vs, 1 / vs).
template <bool MASKED>
__device__ __forceinline__ float softmax_tile(float (&s)[128], uint32_t (&P)[64], int valid, float rowf, const float4* sc,
                                              float& m_ref, float& alpha, bool& need) {
  float a[4], lv[4], rv[4], mt = -INFINITY;
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const float4 v = sc[c];
    a[c] = v.x * rowf;
    lv[c] = v.y;
    rv[c] = v.z;
    if (MASKED) {
#pragma unroll
      for (int i = 0; i < 32; ++i)
        if (32 * c + i >= valid) s[32 * c + i] = -INFINITY;
    }
    float m = max3(s[32 * c], s[32 * c + 1], s[32 * c + 2]);
#pragma unroll
    for (int i = 3; i + 1 < 32; i += 2) m = max3(m, s[32 * c + i], s[32 * c + i + 1]);
    m = fmaxf(m, s[32 * c + 31]);
    mt = fmaxf(mt, fmaf(m, a[c], lv[c]));
  }
  need = mt > m_ref + LA_CACHE_P_TAU;
  const float mn = need ? mt : m_ref;
  alpha = need ? fast_exp2(m_ref - mn) : 1.0f;
  m_ref = mn;
  const float base = LA_CACHE_P_BIAS - (mn == -INFINITY ? 0.f : mn);
  float l = 0.f;
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const float2 aa = make_float2(a[c], a[c]), off = make_float2(base + lv[c], base + lv[c]);
    float2 acc[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int j = 16 * c + i;
      const float2 x = __ffma2_rn(make_float2(s[2 * j], s[2 * j + 1]), aa, off);
      float2 p = make_float2(fast_exp2(x.x), fast_exp2(x.y));
      if (MASKED) {                          // a masked key is 0, whatever its page's scale
        if (2 * j >= valid) p.x = 0.f;
        if (2 * j + 1 >= valid) p.y = 0.f;
      }
      acc[i & 1] = __fadd2_rn(acc[i & 1], p);
      P[j] = pack_f16x2(p.x, p.y);
    }
    const float2 t = __fadd2_rn(acc[0], acc[1]);
    const float sum = t.x + t.y;
    if (!MASKED || 32 * c < valid) l = fmaf(sum, rv[c], l);
  }
  return l;
}

template <typename T, int D>
__global__ void __launch_bounds__(THREADS, 1)
k_attn_cache_tc(const __grid_constant__ AttnCacheParams p) {
  constexpr uint32_t TILE = tile_bytes<D>();
  constexpr int NS = stages<D>();
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = smem;                       // Q_A, Q_B
  uint8_t* sK = smem + 2 * TILE;            // NS tiles
  uint8_t* sV = sK + NS * TILE;
  float4* sS = reinterpret_cast<float4*>(sV + NS * TILE);          // [NSC][4]
  uint64_t* bars = reinterpret_cast<uint64_t*>(sS + NSC * 4);
  uint64_t* q_full = bars;
  uint64_t* k_full = bars + 1;
  uint64_t* v_full = k_full + NS;
  uint64_t* k_empty = v_full + NS;
  uint64_t* v_empty = k_empty + NS;
  uint64_t* sc_full = v_empty + NS;         // [NSC]
  uint64_t* s_full = sc_full + NSC;         // [2]
  uint64_t* p_full = s_full + 2;            // [2]
  uint64_t* pv_done = p_full + 2;           // [2]
  uint64_t* drain = pv_done + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  __shared__ volatile int abort_flag;

  if (p.nsplit > 1) launch_dependents();
  const int b = blockIdx.z, hk = blockIdx.y;
  const int split = blockIdx.x % p.nsplit;
  const int pair = gridDim.x / p.nsplit - 1 - blockIdx.x / p.nsplit;   // under a causal mask the last rows have the most keys
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const CacheSeq s = cache_seq(p, b);
  if (s.bad && blockIdx.x == 0 && hk == 0 && threadIdx.x == 0) raise_device_error(p.err, LA_DEVERR_BAD_DESC);
  const int G = p.heads / p.kv_heads;
  const long long rows = static_cast<long long>(s.n) * G;
  const long long r0 = pair * 256LL;
  if (r0 >= rows) return;
  const int nq = r0 + 128 < rows ? 2 : 1;
  const long long last = min(rows, r0 + 256) - 1;
  const int keys = cache_limit(p, s, static_cast<int>(last / G));      // limits do not fall along the rows
  const int tiles = (keys + 127) / 128;
  const int per = (tiles + p.nsplit - 1) / p.nsplit;
  const int t0 = min(split * per, tiles);
  const int nt = min(tiles, t0 + per) - t0;
  int* err = p.err;

  if (threadIdx.x == 0) {
    abort_flag = 0;
    mbar_init(q_full, 8);
    for (int i = 0; i < NS; ++i) {
      mbar_init(&k_full[i], 4);
      mbar_init(&v_full[i], 4);
      mbar_init(&k_empty[i], 1);
      mbar_init(&v_empty[i], 1);
    }
    for (int i = 0; i < NSC; ++i) mbar_init(&sc_full[i], 1);
    for (int w = 0; w < 2; ++w) {
      mbar_init(&s_full[w], 1);
      mbar_init(&p_full[w], 4);
      mbar_init(&pv_done[w], 1);
    }
    mbar_init(drain, 1);
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp < 4) {
    regs_dec<REGS_LOW>();
    if (warp == 1) {
      // -------------------------------------------------------------- MMA issuer
      auto wwait = [&](uint64_t* bar, uint32_t par) { return __all_sync(0xffffffffu, mbar_wait(bar, par, err)); };
      constexpr uint32_t idS = idesc_fp16(128, 128, false, false);
      constexpr uint32_t idPV = idesc_fp16(128, D, false, true);
      const uint64_t dQ = sdesc_kmajor(smem_u32(sQ));
      const uint64_t dK = sdesc_kmajor(smem_u32(sK));
      const uint64_t dV = sdesc_mnmajor(smem_u32(sV), BOX);
      auto issue_s = [&](int w, uint32_t st) {
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = (kk >> 2) * BOX + (kk & 3) * 32;
          umma_bf16_ss(tmem + s_col(w), dQ + ((w * TILE + off) >> 4), dK + ((st * TILE + off) >> 4), idS, kk > 0 ? 1u : 0u);
        }
        umma_commit(&s_full[w]);
      };
      bool ok = nt == 0 || (wwait(q_full, 0) && wwait(&k_full[0], 0));
      if (ok && nt > 0) {
        tc_fence_after();
        if (elect_one()) {
          for (int w = 0; w < nq; ++w) issue_s(w, 0);
          umma_commit(&k_empty[0]);
        }
        __syncwarp();
      }
      for (int t = 0; t < nt && ok; ++t) {
        const bool more = t + 1 < nt;
        const uint32_t vs = t % NS, vpar = (t / NS) & 1, ks = (t + 1) % NS, kpar = ((t + 1) / NS) & 1;
        ok = wwait(&v_full[vs], vpar) && (!more || wwait(&k_full[ks], kpar));
        for (int w = 0; w < nq && ok; ++w) {
          if (!wwait(&p_full[w], static_cast<uint32_t>(t & 1))) { ok = false; break; }
          tc_fence_after();
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)
              umma_bf16_ts(tmem + o_col(w), tmem + s_col(w) + kk * 8, dV + ((vs * TILE + kk * 2048) >> 4), idPV,
                           (t > 0 || kk > 0) ? 1u : 0u);
            if (more) issue_s(w, ks);
            else umma_commit(&pv_done[w]);
          }
          __syncwarp();
        }
        if (!ok) break;
        if (elect_one()) {
          umma_commit(&v_empty[vs]);
          if (more) umma_commit(&k_empty[ks]);
        }
        __syncwarp();
      }
      if (!ok) abort_flag = 1;
      if (elect_one()) umma_commit(drain);
      __syncwarp();
      wwait(drain, 0);
    }
  } else if (warp >= 12) {
    // ---------------------------------------------------------------- K and V
    regs_dec<REGS_LOAD>();
    constexpr int CH = D / 64;               // 16-byte chunks of a row a lane takes
    const int lw = warp - 12;
    const int row = lw * 8 + (lane & 7);     // + 32 i
    const int ch = lane >> 3;                // + 4 j
    uint4 kb[4][CH], vb[4][CH];
    int pg[4], pgn[4];
    auto find = [&](int t, int (&x)[4]) {    // pages of the tile's four 32-key chunks
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int key = (t0 + t) * 128 + 32 * i;
        x[i] = t < nt && key < keys ? cache_page(p, b, key) : -1;
      }
    };
    auto load = [&](const uint8_t* pages, int t, const int (&x)[4], uint4 (&buf)[4][CH]) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int key = (t0 + t) * 128 + 32 * i + row;
        const bool on = x[i] >= 0 && key < keys;            // rows behind the last key are zeros
        const uint8_t* src = pages + (static_cast<long long>(on ? x[i] : 0) * p.kv_heads + hk) * (p.page_tokens * D) +
                             (key & (p.page_tokens - 1)) * D + ch * 16;
#pragma unroll
        for (int j = 0; j < CH; ++j)
          buf[i][j] = on ? __ldg(reinterpret_cast<const uint4*>(src + j * 64)) : make_uint4(0, 0, 0, 0);
      }
    };
    auto store = [&](uint8_t* tile, const uint4 (&buf)[4][CH]) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = 32 * i + row;
#pragma unroll
        for (int j = 0; j < CH; ++j) {
          const uint4 w = buf[i][j];
          uint8_t* dst = tile + j * BOX + r * 128;           // chunk ch + 4 j: box j, fp16 chunks 2 ch and 2 ch + 1
          *reinterpret_cast<uint4*>(dst + (((2 * ch) ^ (r & 7)) << 4)) =
              make_uint4(e4m3x2_f16x2_lo(w.x), e4m3x2_f16x2_hi(w.x), e4m3x2_f16x2_lo(w.y), e4m3x2_f16x2_hi(w.y));
          *reinterpret_cast<uint4*>(dst + (((2 * ch + 1) ^ (r & 7)) << 4)) =
              make_uint4(e4m3x2_f16x2_lo(w.z), e4m3x2_f16x2_hi(w.z), e4m3x2_f16x2_lo(w.w), e4m3x2_f16x2_hi(w.w));
        }
      }
    };
    auto hand = [&](uint64_t* bar) {
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar);
    };
    if (nt > 0) {
      find(0, pg);
      load(p.k_pages, 0, pg, kb);
      load(p.v_pages, 0, pg, vb);
    }
    for (int t = 0; t < nt && !abort_flag; ++t) {
      const uint32_t st = t % NS, par = (t / NS) & 1;
      find(t + 1, pgn);
      if (lw == 0) {
        // The slot was last read by the softmax of tile t - NSC.  That has ended: this
        // K stage was freed by the scores of tile t - NS, which were issued behind the
        // P of tile t - NS - 1 >= t - NSC.
        if (!mbar_wait(&k_empty[st], par ^ 1, err)) { abort_flag = 1; break; }
        if (lane < 4) {
          const int key = (t0 + t) * 128 + 32 * lane;
          const int x = lane == 0 ? pg[0] : lane == 1 ? pg[1] : lane == 2 ? pg[2] : pg[3];
          float4 v = make_float4(1.f, -INFINITY, 0.f, 0.f);   // keys of no page are not seen
          if (x >= 0 && key < keys) {
            const long long plane = static_cast<long long>(x) * p.kv_heads + hk;
            const float vs = __ldg(p.v_scale + plane);
            v = make_float4(__ldg(p.k_scale + plane), log2f(vs), 1.0f / vs, 0.f);
          }
          sS[(t % NSC) * 4 + lane] = v;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sc_full[t % NSC]);
      } else if (!mbar_wait(&k_empty[st], par ^ 1, err)) {
        abort_flag = 1;
        break;
      }
      store(sK + st * TILE, kb);
      hand(&k_full[st]);
      if (t + 1 < nt) load(p.k_pages, t + 1, pgn, kb);
      if (!mbar_wait(&v_empty[st], par ^ 1, err)) { abort_flag = 1; break; }
      store(sV + st * TILE, vb);
      hand(&v_full[st]);
      if (t + 1 < nt) load(p.v_pages, t + 1, pgn, vb);
#pragma unroll
      for (int i = 0; i < 4; ++i) pg[i] = pgn[i];
    }
  } else {
    // ---------------------------------------------------------------- softmax
    regs_inc<REGS_SOFT>();
    const int w = (warp >> 2) - 1;
    const int quarter = warp & 3;
    const int r = quarter * 32 + lane;
    const long long rr = r0 + w * 128 + r;
    const bool on = rr < rows;
    const int tok = s.q0 + static_cast<int>((on ? rr : 0) / G), head = hk * G + static_cast<int>((on ? rr : 0) % G);
    const int lim = on ? cache_limit(p, s, static_cast<int>(rr / G)) : 0;
    float rowf;
    {
      const T* q = static_cast<const T*>(p.q) + tok * p.q_st + head * p.q_sh;
      uint8_t* dst = sQ + w * TILE + r * 128;
      uint32_t amax = 0;
      auto each = [&](auto&& f) {            // f(chunk of 8, its values)
        if (p.q_vec) {
#pragma unroll 4
          for (int c = 0; c < D / 8; ++c) {
            uint4 u = make_uint4(0, 0, 0, 0);
            if (on) u = __ldg(reinterpret_cast<const uint4*>(q) + c);
            const T* e = reinterpret_cast<const T*>(&u);
            float v[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = q_to_f32(e[k]);
            f(c, v);
          }
        } else {
#pragma unroll 1
          for (int c = 0; c < D / 8; ++c) {
            float v[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = on ? q_to_f32(q[8 * c + k]) : 0.f;
            f(c, v);
          }
        }
      };
      each([&](int, const float (&v)[8]) {
#pragma unroll
        for (int k = 0; k < 8; ++k) amax = max(amax, __float_as_uint(v[k]) & 0x7fffffffu);
      });
      const float g = q_row_scale(amax);
      rowf = p.scale_log2 / g;
      each([&](int c, const float (&v)[8]) {
        *reinterpret_cast<uint4*>(dst + (c >> 3) * BOX + (((c & 7) ^ (r & 7)) << 4)) =
            make_uint4(pack_f16x2(v[0] * g, v[1] * g), pack_f16x2(v[2] * g, v[3] * g), pack_f16x2(v[4] * g, v[5] * g),
                       pack_f16x2(v[6] * g, v[7] * g));
      });
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(q_full);
    }
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t s_base = tmem + lane_off + s_col(w);
    const uint32_t o_base = tmem + lane_off + o_col(w);
    if (w < nq) {
      float m_ref = -INFINITY, l = 0.f;
      bool ok = true;
      for (int t = 0; t < nt; ++t) {
        const int valid = lim - (t0 + t) * 128;
        if (abort_flag || !mbar_wait(&sc_full[t % NSC], static_cast<uint32_t>((t / NSC) & 1), err) ||
            !mbar_wait(&s_full[w], static_cast<uint32_t>(t & 1), err)) {
          ok = false;
          break;
        }
        tc_fence_after();
        float sv[128];
        {
          uint32_t u[4][32];
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_ld32(s_base + c * 32, u[c]);
          tmem_ld_wait();
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int i = 0; i < 32; ++i) sv[32 * c + i] = __uint_as_float(u[c][i]);
        }
        uint32_t P[64];
        float alpha;
        bool need;
        const float4* sc = sS + (t % NSC) * 4;
        const float rs = __all_sync(0xffffffffu, valid >= 128)
                             ? softmax_tile<false>(sv, P, valid, rowf, sc, m_ref, alpha, need)
                             : softmax_tile<true>(sv, P, valid, rowf, sc, m_ref, alpha, need);
        if (t >= 1 && __any_sync(0xffffffffu, need)) {
          // O is stable: the commit that signalled S(t) also covers PV(t-1), issued before it
#pragma unroll 1
          for (int c4 = 0; c4 < D / 32; ++c4) {
            uint32_t o[32];
            tmem_ld32(o_base + c4 * 32, o);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
            tmem_st32(o_base + c4 * 32, o);
          }
        }
        tmem_st32(s_base, *reinterpret_cast<uint32_t(*)[32]>(P));
        tmem_st32(s_base + 32, *reinterpret_cast<uint32_t(*)[32]>(P + 32));
        tmem_st_wait();
        l = l * alpha + rs;
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[w]);
      }
      if (!ok) abort_flag = 1;
      const long long part = (static_cast<long long>(split) * p.tokens + tok) * p.heads + head;
      if (ok && (nt == 0 || mbar_wait(&pv_done[w], 0, err))) {
        tc_fence_after();
        if (p.nsplit > 1 && on) p.part_ml[part] = make_float2(m_ref, l);
#pragma unroll 1
        for (int c4 = 0; c4 < D / 32; ++c4) {
          uint32_t o[32];
          if (nt > 0) {
            tmem_ld32(o_base + c4 * 32, o);
            tmem_ld_wait();
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = 0;
          }
          if (on) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float v[4] = {__uint_as_float(o[4 * i]), __uint_as_float(o[4 * i + 1]), __uint_as_float(o[4 * i + 2]),
                                  __uint_as_float(o[4 * i + 3])};
              if (p.nsplit > 1)
                *reinterpret_cast<float4*>(p.part_o + part * D + c4 * 32 + 4 * i) = make_float4(v[0], v[1], v[2], v[3]);
              else
                cache_store4<T>(p, tok, head, c4 * 32 + 4 * i, v, l);
            }
          }
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, TMEM_COLS);
  }
}

template <typename T, int D>
cudaError_t launch(const AttnCacheParams& p, cudaStream_t st) {
  auto kern = k_attn_cache_tc<T, D>;
  constexpr size_t SMEM = smem_bytes<D>();
  // The register split assumes exactly LAUNCH_REGS registers a thread at launch.
  static const int regs = [&] {
    cudaFuncAttributes fa{};
    return cudaFuncGetAttributes(&fa, kern) == cudaSuccess ? fa.numRegs : -1;
  }();
  if (regs != LAUNCH_REGS) {
    std::fprintf(stderr, "k_attn_cache_tc: compiled with %d registers a thread, the register split needs %d\n", regs,
                 LAUNCH_REGS);
    return cudaErrorInvalidConfiguration;
  }
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(SMEM));
  if (e != cudaSuccess) return e;
  const long long rows = static_cast<long long>(p.max_q) * (p.heads / p.kv_heads);
  const long long gx = (rows + 255) / 256 * p.nsplit;
  if (gx > 0x7fffffffLL) return cudaErrorInvalidValue;
  kern<<<dim3(static_cast<unsigned>(gx), p.kv_heads, p.batch), THREADS, SMEM, st>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attn_cache_tc(int dtype, const AttnCacheParams& p, cudaStream_t st) {
  if (dtype == LA_BF16) return p.d == 64 ? launch<__nv_bfloat16, 64>(p, st) : launch<__nv_bfloat16, 128>(p, st);
  return p.d == 64 ? launch<__half, 64>(p, st) : launch<__half, 128>(p, st);
}
