// la_op_attention_cache_fp8 for many query rows of a key head: tcgen05 (kind::f16),
// two 128-row tiles a CTA.
//
// One CTA = up to 256 rows (query token x head of the key head's group) of one
// sequence and key head, over one piece of the keys in tiles of 128.  16 warps:
//   warp 0       looks up pages and scales and brings the codes: one bulk copy (TMA)
//                per page and tile, since a page's head is one run of bytes
//   warp 1       owns tensor memory (512 columns: S_A | S_B | O_A | O_B) and issues
//                the MMAs: PV_A(t), S_A(t+1), PV_B(t), S_B(t+1), ..., so that one
//                tile's softmax runs beside the other's products; warps 2, 3 idle
//   warps 4-11   softmax of tiles A and B, a thread a row; before that they bring Q
//                to shared memory as fp16 under a power of two per row
//   warps 12-15  unpack a tile's codes into fp16 (exactly), in the 128-byte-swizzled
//                layout that the MMAs read, and hand it to them in a ring
// The codes are unpacked once for 256 rows; at 64 conversions a clock and SM that
// takes a quarter of the tile's MMA time and runs beside it.  fp16 operands keep q
// and the codes exact and P to 11 bits (e4m3 or bf16 P would not).  Threads that
// loaded the codes themselves lost more than they saved: the proxy fence behind each
// tile waits for the loads that are under way for the next one (1.96 ms against
// 1.57 ms at 4680 x 15600 x 40 x 128).
//
// Scales: the score of a key is acc * ks * (row factor); log2(vs) enters the
// exponent, so a page's P carries its value scale and the normaliser takes it out
// again (sum * 1 / vs): scales cost no instruction an element beyond the scale and
// offset that the exponent needs anyway.  A tile with a page whose value scale lies far
// below an earlier one (see LA_CACHE_SPREAD) gets 0 for 1 / vs, and its weights are
// summed by themselves, without the scales; the others pay 0 to 2 % for the question
// (2 x 4680 q x 7800 keys x 16 heads, frame-causal: 600 us a call, 590 without).
//
// Waits are bounded.  Lanes of a warp may see one end differently (each looks at the
// clock and at the CTA's abort flag by itself), and what follows needs all of them, so
// every answer is put to a vote (602 us for the same case).
#include <cstdio>

#include "attn_cache.cuh"

namespace {

constexpr int THREADS = 512;
constexpr int LAUNCH_REGS = 128;            // 65536 / 512
constexpr int REGS_LOW = 96;                // warps 0-3
constexpr int REGS_LOAD = 96;               // warps 12-15
constexpr int REGS_SOFT = 160;              // warps 4-11
static_assert(128 * (REGS_LOW + REGS_LOAD + 2 * REGS_SOFT) <= THREADS * LAUNCH_REGS, "register split exceeds the launch");
constexpr uint32_t BOX = 16384;             // 128 rows x 64 fp16, 128-byte swizzle
constexpr uint32_t TMEM_COLS = 512;
constexpr int NSC = 8;                      // ring of the tiles' scales
static_assert(NSC >= 4 + 2, "the scales outlast the K ring and the tile of codes before it");

template <int D> __host__ __device__ constexpr uint32_t tile_bytes() { return D / 64 * BOX; }
template <int D> __host__ __device__ constexpr int stages() { return D == 64 ? 4 : 2; }
// Parts in which a tile's P is handed to the tensor core.
template <int D> __host__ __device__ constexpr int hands() { return D == 64 ? 2 : 1; }
template <int D> __host__ __device__ constexpr size_t smem_bytes() {
  return 1024 + 2 * tile_bytes<D>() + stages<D>() * 2 * tile_bytes<D>() + 2 * 128 * D + NSC * 64 + 512;
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

// Bytes from global to shared memory (16-byte aligned, a multiple of 16), counted on bar.
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
               ::"r"(smem_u32(dst)), "l"(src), "r"(bytes), "r"(smem_u32(bar)) : "memory");
}

// Waits for this warp's tensor-memory loads; u is used behind it only.
__device__ __forceinline__ void ld_wait(uint32_t (&u)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(u[0]), "+r"(u[1]), "+r"(u[2]), "+r"(u[3]), "+r"(u[4]), "+r"(u[5]), "+r"(u[6]), "+r"(u[7]), "+r"(u[8]),
                 "+r"(u[9]), "+r"(u[10]), "+r"(u[11]), "+r"(u[12]), "+r"(u[13]), "+r"(u[14]), "+r"(u[15]), "+r"(u[16]),
                 "+r"(u[17]), "+r"(u[18]), "+r"(u[19]), "+r"(u[20]), "+r"(u[21]), "+r"(u[22]), "+r"(u[23]), "+r"(u[24]),
                 "+r"(u[25]), "+r"(u[26]), "+r"(u[27]), "+r"(u[28]), "+r"(u[29]), "+r"(u[30]), "+r"(u[31])::"memory");
}

// The running maximum of a row over a key tile's scores (raw accumulators in tensor
// memory, log2 domain with the value scale); root: the square root of the factor that
// takes sums from the old one to it.  sc[c]: a 32-key chunk's (ks, log2 vs, 1 / vs).
// The scores are read twice, 32 at a time, once here: 128 of them held at once would not
// fit beside the other warps' registers.
template <bool MASKED>
__device__ __forceinline__ void softmax_max(uint32_t s_base, int valid, float rowf, const float4* sc, float& m_ref,
                                            float& root) {
  uint32_t u[2][32];
  float mt = -INFINITY;
  tmem_ld32(s_base, u[0]);
  ld_wait(u[0]);
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    if (c < 3) tmem_ld32(s_base + (c + 1) * 32, u[(c + 1) & 1]);
    float m[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float x[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        x[i] = __uint_as_float(u[c & 1][8 * k + i]);
        if (MASKED && 32 * c + 8 * k + i >= valid) x[i] = -INFINITY;
      }
      m[k] = max3(max3(x[0], x[1], x[2]), max3(x[3], x[4], x[5]), fmaxf(x[6], x[7]));
    }
    const float2 v = *reinterpret_cast<const float2*>(sc + c);
    mt = fmaxf(mt, fmaf(max3(fmaxf(m[0], m[1]), m[2], m[3]), v.x * rowf, v.y));
    if (c < 3) ld_wait(u[(c + 1) & 1]);
  }
  const bool need = mt > m_ref + LA_CACHE_P_TAU;
  const float mn = need ? mt : m_ref;
  root = need ? fast_exp2(0.5f * (m_ref - mn)) : 1.0f;
  m_ref = mn;
}

// The row's share of a tile in the normaliser, straight from the scores.
__device__ __forceinline__ float softmax_sum(uint32_t s_base, int valid, float rowf, const float4* sc, float m_ref) {
  const float base = LA_CACHE_P_BIAS - (m_ref == -INFINITY ? 0.f : m_ref);
  float l = 0.f;
#pragma unroll 1
  for (int c = 0; c < 4; ++c) {
    uint32_t u[32];
    tmem_ld32(s_base + c * 32, u);
    ld_wait(u);
    const float4 v = sc[c];
    const float a = v.x * rowf;
    const int n = v.w == 0.f ? 0 : valid - 32 * c;             // keys of no page are not seen
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      const float h = fast_exp2(0.5f * fmaf(__uint_as_float(u[i]), a, base));
      if (i < n) l += h * h;
    }
  }
  return l;
}

// The row's P (fp16 pairs) of 64 keys, chunks c0 and c0 + 1, stored over scores that both
// passes have read by then (P of chunk c lies in chunk c / 2 of the scores), and their
// share of the normaliser.
template <bool MASKED>
__device__ __forceinline__ float softmax_exp(uint32_t s_base, int c0, int valid, float rowf, const float4* sc, float m_ref) {
  uint32_t u[2][32];
  const float base = LA_CACHE_P_BIAS - (m_ref == -INFINITY ? 0.f : m_ref);
  float l = 0.f;
  tmem_ld32(s_base + c0 * 32, u[0]);
  tmem_ld32(s_base + c0 * 32 + 32, u[1]);
  ld_wait(u[0]);
  ld_wait(u[1]);
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int c = c0 + k;
    const float4 v = sc[c];
    const float a = v.x * rowf;
    const float2 aa = make_float2(a, a), off = make_float2(base + v.y, base + v.y);
    float2 acc[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
    uint32_t P[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float2 x = __ffma2_rn(make_float2(__uint_as_float(u[k][2 * i]), __uint_as_float(u[k][2 * i + 1])), aa, off);
      float2 e = make_float2(fast_exp2(x.x), fast_exp2(x.y));
      if (MASKED) {                            // a masked key is 0, whatever its page's scale
        if (32 * c + 2 * i >= valid) e.x = 0.f;
        if (32 * c + 2 * i + 1 >= valid) e.y = 0.f;
      }
      acc[i & 1] = __fadd2_rn(acc[i & 1], e);
      P[i] = pack_f16x2(e.x, e.y);
    }
    const float2 t = __fadd2_rn(acc[0], acc[1]);
    if (!MASKED || 32 * c < valid) l = fmaf(t.x + t.y, v.z, l);
    tmem_st16(s_base + 16 * c, P);
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
  uint8_t* raw = sV + NS * TILE;            // a tile's K codes, then its V codes
  float4* sS = reinterpret_cast<float4*>(raw + 2 * 128 * D);       // [NSC][4] (ks, log2 vs, 1 / vs, page found)
  uint64_t* bars = reinterpret_cast<uint64_t*>(sS + NSC * 4);
  uint64_t* q_full = bars;
  uint64_t* k_full = bars + 1;
  uint64_t* v_full = k_full + NS;
  uint64_t* k_empty = v_full + NS;
  uint64_t* v_empty = k_empty + NS;
  uint64_t* sc_full = v_empty + NS;         // [NSC]
  uint64_t* raw_full = sc_full + NSC;       // K, V
  uint64_t* raw_empty = raw_full + 2;       // K, V
  uint64_t* s_full = raw_empty + 2;         // [2]
  uint64_t* p_full = s_full + 2;            // [tile][half of its keys]
  uint64_t* pv_done = p_full + 4;           // [2]
  uint64_t* drain = pv_done + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  __shared__ volatile int abort_flag;

  if (p.nsplit > 1) launch_dependents();
  const int cta = blockIdx.x;
  const bool whole = cta < p.full;              // else one of the unit's nsplit pieces
  const int unit = whole ? cta : p.full + (cta - p.full) / p.nsplit;
  const int split = whole ? 0 : (cta - p.full) % p.nsplit, nsplit = whole ? 1 : p.nsplit;
  const CacheUnit at_unit = cache_unit(p, unit);
  const int b = at_unit.b, hk = at_unit.hk, pair = at_unit.pair;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const CacheSeq s = cache_seq(p, b);
  if (s.bad && pair == 0 && split == 0 && hk == 0 && threadIdx.x == 0) raise_device_error(p.err, LA_DEVERR_BAD_DESC);
  const int G = p.heads / p.kv_heads;
  const long long rows = static_cast<long long>(s.n) * G;
  const long long r0 = pair * 256LL;
  if (r0 >= rows) return;
  const int nq = r0 + 128 < rows ? 2 : 1;
  const long long last = min(rows, r0 + 256) - 1;
  const int keys = cache_limit(p, s, static_cast<int>(last / G));      // limits do not fall along the rows
  const int tiles = (keys + 127) / 128;
  const int per = (tiles + nsplit - 1) / nsplit;
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
      mbar_init(&raw_full[w], 1);
      mbar_init(&raw_empty[w], 4);
      mbar_init(&s_full[w], 1);
      mbar_init(&p_full[2 * w], 4);
      mbar_init(&p_full[2 * w + 1], 4);
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
    if (warp == 0) {
      // ------------------------------------------------------------ pages, scales, codes
      // Lane c < 4 has the tile's 32-key chunk c, and copies for its page if the page
      // (or the tile's part of it) starts there.
      const int span = min(128, p.page_tokens);
      int t = 0;
      bool ok = true;
      float top_lv = -INFINITY;
      for (; t < nt && ok; ++t) {
        const int key = (t0 + t) * 128 + 32 * lane;
        int pg = -1;
        float4 v = make_float4(1.f, -INFINITY, 0.f, 0.f);     // keys of no page are not seen
        long long plane = 0;
        uint32_t bytes = 0;
        if (lane < 4 && key < keys) {
          pg = cache_page(p, b, key);
          if (pg >= 0) {
            plane = static_cast<long long>(pg) * p.kv_heads + hk;
            const float vs = __ldg(p.v_scale + plane);
            v = make_float4(__ldg(p.k_scale + plane), log2f(vs), 1.0f / vs, 1.f);
            if ((32 * lane) % span == 0) bytes = static_cast<uint32_t>(min(span, keys - key)) * D;
          }
        }
        float low = pg >= 0 ? v.y : INFINITY;
        top_lv = fmaxf(top_lv, pg >= 0 ? v.y : -INFINITY);
#pragma unroll
        for (int o = 1; o < 4; o *= 2) {
          low = fminf(low, __shfl_xor_sync(0xffffffffu, low, o));
          top_lv = fmaxf(top_lv, __shfl_xor_sync(0xffffffffu, top_lv, o));
        }
        // a tile whose first page is not there is summed in that way, too
        const int first = __shfl_sync(0xffffffffu, pg, 0);
        if (first < 0 || low < top_lv - LA_CACHE_SPREAD) v.z = 0.f;
        uint32_t all = bytes;
        all += __shfl_xor_sync(0xffffffffu, all, 1);
        all += __shfl_xor_sync(0xffffffffu, all, 2);
        const long long at = plane * (p.page_tokens * D) + (key & (p.page_tokens - 1)) * D;
        // The scales' slot was last read by the softmax of tile t - NSC, which has ended:
        // the codes of tile t - 1 were unpacked into a K stage that the scores of tile
        // t - 1 - NS freed, which were issued behind the P of tile t - 2 - NS >= t - NSC.
        for (int i = 0; i < 2 && ok; ++i) {
          ok = __all_sync(0xffffffffu, !abort_flag && mbar_wait(&raw_empty[i], (t & 1) ^ 1, err));
          if (!ok) break;
          if (i == 0 && lane < 4) sS[(t % NSC) * 4 + lane] = v;
          __syncwarp();
          if (lane == 0) {
            if (i == 0) mbar_arrive(&sc_full[t % NSC]);
            mbar_expect_tx(&raw_full[i], all);
          }
          __syncwarp();
          if (bytes) bulk_load(raw + i * 128 * D + 32 * lane * D, (i ? p.v_pages : p.k_pages) + at, bytes, &raw_full[i]);
        }
      }
      // No copy may land behind the CTA's end.  After an error (t - 1 is the tile that
      // was given up) a wait for a copy that was never started ends at its limit.
      for (int i = 0; i < 2 && t > 0; ++i) {
        if (!ok && t > 1) mbar_wait(&raw_full[i], t & 1, err);
        mbar_wait(&raw_full[i], (t - 1) & 1, err);
      }
    } else if (warp == 1) {
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
#pragma unroll
          for (int h = 0; h < hands<D>(); ++h) {
            ok = ok && wwait(&p_full[2 * w + h], static_cast<uint32_t>(t & 1));
            if (!ok) break;
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
              for (int kk = h * (8 / hands<D>()); kk < (h + 1) * (8 / hands<D>()); ++kk)
                umma_bf16_ts(tmem + o_col(w), tmem + s_col(w) + kk * 8, dV + ((vs * TILE + kk * 2048) >> 4), idPV,
                             (t > 0 || kk > 0) ? 1u : 0u);
              if (h == hands<D>() - 1) {
                if (more) issue_s(w, ks);
                else umma_commit(&pv_done[w]);
              }
            }
            __syncwarp();
          }
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
    // ---------------------------------------------------------------- unpack
    regs_dec<REGS_LOAD>();
    const int lw = warp - 12;
    // A quarter warp reads 128 bytes of codes in a row's length and writes 8 different
    // 16-byte columns: at D = 128 half a row r and the other half of row r ^ 1.
    const int q8 = lane & 7, cc = q8 & 3, hi = q8 >> 2;
    auto unpack = [&](const uint8_t* codes, uint8_t* tile, int t) {
      const float4* sc = sS + (t % NSC) * 4;
      const int left = keys - (t0 + t) * 128;              // rows behind the last key become zeros
#pragma unroll 2
      for (int i = 0; i < D / 16; ++i) {
        const int r0 = i * 16 + lw * 4 + (lane >> 3);
        const int r = D == 128 ? r0 ^ hi : 2 * r0 + hi;
        const int box = D == 128 ? hi : 0;
        uint4 w = *reinterpret_cast<const uint4*>(codes + r * D + box * 64 + cc * 16);
        if (r >= left || sc[r >> 5].w == 0.f) w = make_uint4(0, 0, 0, 0);
        uint8_t* dst = tile + box * BOX + r * 128;
        *reinterpret_cast<uint4*>(dst + (((2 * cc) ^ (r & 7)) << 4)) =
            make_uint4(e4m3x2_f16x2_lo(w.x), e4m3x2_f16x2_hi(w.x), e4m3x2_f16x2_lo(w.y), e4m3x2_f16x2_hi(w.y));
        *reinterpret_cast<uint4*>(dst + (((2 * cc + 1) ^ (r & 7)) << 4)) =
            make_uint4(e4m3x2_f16x2_lo(w.z), e4m3x2_f16x2_hi(w.z), e4m3x2_f16x2_lo(w.w), e4m3x2_f16x2_hi(w.w));
      }
    };
    for (int t = 0; t < nt; ++t) {
      const uint32_t st = t % NS, par = (t / NS) & 1;
      bool ok = true;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        ok = __all_sync(0xffffffffu, !abort_flag && mbar_wait(&raw_full[i], t & 1, err) &&
                                         mbar_wait(i ? &v_empty[st] : &k_empty[st], par ^ 1, err));
        if (!ok) break;
        unpack(raw + i * 128 * D, (i ? sV : sK) + st * TILE, t);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(i ? &v_full[st] : &k_full[st]);
          mbar_arrive(&raw_empty[i]);
        }
      }
      if (!ok) { abort_flag = 1; break; }
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
      uint4 raw_q[D / 8];                    // the row, all of it under way at once
#pragma unroll
      for (int c = 0; c < D / 8; ++c) {
        raw_q[c] = make_uint4(0, 0, 0, 0);
        if (on && p.q_vec) raw_q[c] = __ldg(reinterpret_cast<const uint4*>(q) + c);
      }
      if (on && !p.q_vec) {
#pragma unroll
        for (int c = 0; c < D / 8; ++c) {
          uint32_t e[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) e[k] = reinterpret_cast<const unsigned short*>(q)[8 * c + k];
          raw_q[c] = make_uint4(e[0] | e[1] << 16, e[2] | e[3] << 16, e[4] | e[5] << 16, e[6] | e[7] << 16);
        }
      }
#pragma unroll
      for (int c = 0; c < D / 8; ++c)
#pragma unroll
        for (int k = 0; k < 8; ++k)
          amax = max(amax, __float_as_uint(q_to_f32(reinterpret_cast<const T*>(&raw_q[c])[k])) & 0x7fffffffu);
      const float g = q_row_scale(amax);
      rowf = p.scale_log2 / g;
#pragma unroll
      for (int c = 0; c < D / 8; ++c) {
        float v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = q_to_f32(reinterpret_cast<const T*>(&raw_q[c])[k]) * g;
        *reinterpret_cast<uint4*>(dst + (c >> 3) * BOX + (((c & 7) ^ (r & 7)) << 4)) =
            make_uint4(pack_f16x2(v[0], v[1]), pack_f16x2(v[2], v[3]), pack_f16x2(v[4], v[5]), pack_f16x2(v[6], v[7]));
      }
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
        ok = __all_sync(0xffffffffu, !abort_flag && mbar_wait(&sc_full[t % NSC], static_cast<uint32_t>((t / NSC) & 1), err) &&
                                         mbar_wait(&s_full[w], static_cast<uint32_t>(t & 1), err));
        if (!ok) break;
        tc_fence_after();
        float root;
        const float4* sc = sS + (t % NSC) * 4;
        const bool full = __all_sync(0xffffffffu, valid >= 128);
        if (full) softmax_max<false>(s_base, valid, rowf, sc, m_ref, root);
        else softmax_max<true>(s_base, valid, rowf, sc, m_ref, root);
        const bool apart = sc->z == 0.f;          // the same in every lane
        if (__any_sync(0xffffffffu, root != 1.0f || apart)) {
          const float alpha = root * root;
          l = l * root * root;
          if (apart) l += softmax_sum(s_base, valid, rowf, sc, m_ref);
          // O is stable: the commit that signalled S(t) also covers PV(t-1), issued before
          // it; the first tile finds nothing in it
#pragma unroll 1
          for (int c4 = t >= 1 ? 0 : D / 32; c4 < D / 32; ++c4) {
            uint32_t o[32];
            tmem_ld32(o_base + c4 * 32, o);
            ld_wait(o);
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
            tmem_st32(o_base + c4 * 32, o);
          }
        }
        // At D = 64 the first half of P is handed over as soon as it is there: its products
        // run beside the second half's exponentials (4 prompts of up to 1013 rows: 113.9
        // us, 114.9 in one).  At D = 128 that is no faster (4680 x 15600 x 40: 1611 us, 1589
        // in one).
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          l += full ? softmax_exp<false>(s_base, 2 * h, valid, rowf, sc, m_ref)
                    : softmax_exp<true>(s_base, 2 * h, valid, rowf, sc, m_ref);
          if (hands<D>() == 1 && h == 0) continue;
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&p_full[2 * w + (hands<D>() == 1 ? 0 : h)]);
        }
      }
      if (!ok) abort_flag = 1;
      const long long part = (static_cast<long long>(split) * (p.units - p.full) + unit - p.full) * 256 + w * 128 + r;
      ok = __all_sync(0xffffffffu, ok && (nt == 0 || mbar_wait(&pv_done[w], 0, err)));
      if (ok) {
        tc_fence_after();
        if (!whole && on) p.part_ml[part] = make_float2(m_ref, l);
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
            for (int i = 0; i < 4; ++i) {
              float v[8];
#pragma unroll
              for (int k = 0; k < 8; ++k) v[k] = __uint_as_float(o[8 * i + k]);
              if (!whole) {
                float4* to = reinterpret_cast<float4*>(p.part_o + part * D + c4 * 32 + 8 * i);
                to[0] = make_float4(v[0], v[1], v[2], v[3]);
                to[1] = make_float4(v[4], v[5], v[6], v[7]);
              } else {
                cache_store8<T>(p, tok, head, c4 * 32 + 8 * i, v, l);
              }
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
  const long long gx = p.full + static_cast<long long>(p.units - p.full) * p.nsplit;
  if (gx > 0x7fffffffLL) return cudaErrorInvalidValue;
  kern<<<static_cast<unsigned>(gx), THREADS, SMEM, st>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attn_cache_tc(int dtype, const AttnCacheParams& p, cudaStream_t st) {
  if (dtype == LA_BF16) return p.d == 64 ? launch<__nv_bfloat16, 64>(p, st) : launch<__nv_bfloat16, 128>(p, st);
  return p.d == 64 ? launch<__half, 64>(p, st) : launch<__half, 128>(p, st);
}
