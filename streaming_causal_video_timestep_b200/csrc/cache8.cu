// la_op_cache_append_fp8: new keys (rotated on the way) and values into pages of
// e4m3 codes with one power-of-two scale for each (page, head).
//
// One CTA takes one page of one sequence, for K or for V, and walks over heads:
// it holds the page's new tokens in registers (fp32, after the rotation), reduces
// their largest magnitude over the CTA, picks the scale and writes the codes, so
// every new element is read once and every code written once.  The next heads'
// elements are on their way meanwhile (cp.async to a ring in shared memory, of which
// each thread reads back what it copied, so nothing waits for another thread but the
// reduction).  Bound: HBM.
//
// An element on the border between two codes goes to one or the other by the last bit of
// its rotation, so that is the fp32 definition's to the bit, as far as the angles are (off
// by |pos| * 2^-60 turns at most): sine and cosine rounded to nearest (in fp64, once for
// all the heads of a CTA), each product and sum rounded by itself.
//
// Scale: 2^k, the smallest with 448 * 2^k >= amax (k >= -64), read off amax's own
// exponent and mantissa, so no rounding decides it.  A page that already holds
// tokens keeps the larger of its scale and that; where it grows, the codes in
// front of the new tokens are multiplied by old / new, a power of two, and rounded
// to e4m3 again: exact but for results below e4m3's normal range.  A magnitude
// that is not finite makes the scale NaN, which marks the page's head until its
// first token is written again.
#include <algorithm>

#include "kernels.h"
#include "rotary.cuh"
#include "sm100.cuh"

namespace {

// Smallest 2^k >= amax / 448 for the bits of amax >= 0: 448 = 1.75 * 2^8.
__device__ __forceinline__ float page_scale(uint32_t amax_bits) {
  if (amax_bits >= 0x7f800000u) return __uint_as_float(0x7fc00000u);
  const int e = static_cast<int>(amax_bits >> 23) - 127;                  // amax = m * 2^e, 1 <= m < 2 (subnormals: clamped)
  const int k = max((amax_bits & 0x7fffffu) <= 0x600000u ? e - 8 : e - 7, -64);
  return __uint_as_float(static_cast<uint32_t>(k + 127) << 23);
}

__device__ __forceinline__ float2 e4m3x2_to_f32(uint32_t two) {
  uint32_t h;
  asm("{\n\t.reg .b16 l, u;\n\tmov.b32 {l, u}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t}" : "=r"(h) : "r"(two));
  return __half22float2(*reinterpret_cast<__half2*>(&h));
}

__device__ __forceinline__ float max_nan3(float a, float b, float c) {
  float d;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

__device__ __forceinline__ void cp_async16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}

// Vectors of the input that a thread holds for one head, and the ring's stages.
template <typename T, int D, int PAGE> struct Ring {
  static constexpr int ALL = PAGE * D / 16;                  // threads that hold a page's head at 16 elements each
  static constexpr int THREADS = ALL < 512 ? ALL : 512;
  static constexpr int NP = ALL / THREADS;
  static constexpr int PER = 16 / Vec16<T>::N;               // 16-byte vectors of 16 elements
  static constexpr int STAGE = NP * PER * THREADS * 16;
  static constexpr int STAGES = STAGE <= 16384 ? 4 : STAGE <= 32768 ? 3 : 2;
};

// A thread owns 16 elements of one token a pass, D/16 threads a row.  VEC: as 16-byte
// vectors, the w-th of thread u at element w * N * D/16 + N * u, so that a row's threads
// read and write next to each other (vectors that lie side by side in a thread fetch
// every 32-byte sector twice), and both elements of a pair are the thread's own: pairs
// lie in a vector, or (HALF: tab.half over all of a row) in vectors half a row apart.
// Not VEC: pairs 8u .. 8u+7.
template <typename T, int D, int PAGE, bool VEC, bool HALF>
__global__ void __launch_bounds__((Ring<T, D, PAGE>::THREADS))
k_cache_append(const __grid_constant__ CacheAppendParams p, const __grid_constant__ RotaryTable tab) {
  using R = Ring<T, D, PAGE>;
  constexpr int THREADS = R::THREADS, NP = R::NP;
  constexpr int TPR = D / 16;                       // threads a row
  constexpr int ROWS = THREADS / TPR;               // rows a pass
  constexpr int N = Vec16<T>::N;
  const int b = blockIdx.x / p.pages_per_seq, at = blockIdx.x % p.pages_per_seq;
  const bool is_v = blockIdx.z != 0;
  const int u = threadIdx.x % TPR, row = threadIdx.x / TPR;

  // The sequence's new tokens, within the arrays whatever the device data says.
  const int c0 = p.cu_new[b], c1 = p.cu_new[b + 1], old_len = p.cache_len[b];
  const long long room = static_cast<long long>(p.max_pages) * PAGE;
  const bool bad = c0 < 0 || c1 < c0 || c1 > p.tokens || old_len < 0 || old_len + static_cast<long long>(c1 - c0) > room ||
                   c1 - c0 > p.max_new;
  if (bad) {
    if (at == 0 && blockIdx.y == 0 && threadIdx.x == 0) raise_device_error(p.err, LA_DEVERR_BAD_DESC);
    return;
  }
  const int page0 = old_len / PAGE + at;            // page of the sequence
  const long long start = max(static_cast<long long>(old_len), static_cast<long long>(page0) * PAGE);
  const long long end = min(static_cast<long long>(old_len) + (c1 - c0), (page0 + 1LL) * PAGE);
  if (start >= end) return;
  const int off0 = static_cast<int>(start - static_cast<long long>(page0) * PAGE);
  const int cnt = static_cast<int>(end - start);
  const int pg = p.block_table[static_cast<long long>(b) * p.max_pages + page0];
  if (pg < 0 || pg >= p.num_pages) {
    if (blockIdx.y == 0 && threadIdx.x == 0) raise_device_error(p.err, LA_DEVERR_BAD_DESC);
    return;
  }
  const long long tok0 = c0 + (start - old_len);    // first new token of the page

  const int h0 = blockIdx.y * p.heads_per_cta, h1 = min(h0 + p.heads_per_cta, p.heads);
  const T* x = static_cast<const T*>(is_v ? p.v : p.k);
  const long long st = is_v ? p.v_st : p.k_st, sh = is_v ? p.v_sh : p.k_sh;
  extern __shared__ __align__(16) uint8_t ring_raw[];
  uint4* ring = reinterpret_cast<uint4*>(ring_raw);
  // This thread's first vector of the next head to fetch, and the stage it goes to.
  const T* src = x + (tok0 + row) * st + h0 * sh + N * u;
  int into = 0;
  auto fetch = [&](int h) {
    if constexpr (VEC) {
      if (h < h1) {
        uint4* to = ring + into * (R::STAGE / 16) + threadIdx.x;
#pragma unroll
        for (int i = 0; i < NP; ++i) {
          if (row + i * ROWS < cnt) {
            const T* xr = src + i * ROWS * st;
#pragma unroll
            for (int w = 0; w < R::PER; ++w) cp_async16(to + (i * R::PER + w) * THREADS, xr + w * (N * TPR));
          }
        }
        src += sh;
        into = into + 1 == R::STAGES ? 0 : into + 1;
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    }
  };
  for (int i = 0; i < R::STAGES - 1; ++i) fetch(h0 + i);

  float2 cs[NP][8];                                 // pairs that are not rotated: (1, 0), exact for finite values
  const bool rotate = !is_v && tab.n > 0;
  if (rotate) {
    __shared__ PairTable pairs;
    pairs.fill(tab);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const int r = row + i * ROWS;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        int j = 8 * u + k;                          // the pair of f[2k], f[2k+1]
        if (VEC && HALF) j = k / N * (N * TPR) + N * u + k % N;               // of f[k], f[k+8]
        else if (VEC) j = (2 * k / N * (N * TPR) + N * u + 2 * k % N) / 2;
        cs[i][k] = r < cnt && j < tab.n ? pairs.cos_sin_nearest(j, p.pos + (tok0 + r) * tab.naxes) : make_float2(1.f, 0.f);
      }
    }
  }
  // The warps' maxima of a head, in turn in one of two rows: a row is written again only
  // behind the barrier of the head between.
  static_assert(THREADS <= 1024, "a row of red holds every warp");
  __shared__ uint32_t red[2][32];
  if (threadIdx.x < 64) red[threadIdx.x / 32][threadIdx.x % 32] = 0;
  __syncthreads();
  int slot = 0, stage = 0;
  uint8_t* pl = (is_v ? p.v_pages : p.k_pages) + (static_cast<long long>(pg) * p.heads + h0) * (PAGE * D);
  float* sc = (is_v ? p.v_scale : p.k_scale) + static_cast<long long>(pg) * p.heads + h0;

  for (int h = h0; h < h1; ++h, ++sc, pl += PAGE * D) {
    if constexpr (VEC) {
      asm volatile("cp.async.wait_group %0;" ::"n"(R::STAGES - 2) : "memory");
      fetch(h + R::STAGES - 1);                     // into the stage that this thread read a head ago
    }
    const uint4* from = ring + stage * (R::STAGE / 16) + threadIdx.x;
    stage = stage + 1 == R::STAGES ? 0 : stage + 1;
    float f[NP][16];
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const int r = row + i * ROWS;
      if (r < cnt) {
        if constexpr (VEC) {
#pragma unroll
          for (int w = 0; w < R::PER; ++w) Vec16<T>::unpack(from[(i * R::PER + w) * THREADS], f[i] + w * N);
        } else {
          const T* xr = x + (tok0 + r) * st + h * sh;
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const int2 e = is_v ? make_int2(16 * u + 2 * k, 16 * u + 2 * k + 1) : pair_elems(tab, 8 * u + k);
            f[i][2 * k] = to_f32(xr[e.x]);
            f[i][2 * k + 1] = to_f32(xr[e.y]);
          }
        }
        if (rotate) {
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            float& a = f[i][VEC && HALF ? k : 2 * k];
            float& b = f[i][VEC && HALF ? k + 8 : 2 * k + 1];
            const float v = a, w = b;
            a = __fsub_rn(__fmul_rn(v, cs[i][k].x), __fmul_rn(w, cs[i][k].y));
            b = __fadd_rn(__fmul_rn(v, cs[i][k].y), __fmul_rn(w, cs[i][k].x));
          }
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) top = max_nan3(top, fabsf(f[i][2 * k]), fabsf(f[i][2 * k + 1]));
      }
    }
    uint32_t amax = __reduce_max_sync(0xffffffffu, __float_as_uint(top));   // bits: NaN > inf > finite
    if (threadIdx.x % 32 == 0) red[slot][threadIdx.x / 32] = amax;
    const float old = off0 ? *sc : 0.f;             // read by every thread before thread 0 writes it
    __syncthreads();
    amax = __reduce_max_sync(0xffffffffu, red[slot][threadIdx.x % 32]);
    slot ^= 1;
    float s = page_scale(amax);
    if (off0) s = (old != old || s != s) ? __uint_as_float(0x7fc00000u) : fmaxf(old, s);
    const bool fine = s == s;
    // 1 / s, a power of two; 0 for the NaN, whose page gets zeros
    // (a scale of another kind can only be the caller's own, from before)
    float inv = fine ? __uint_as_float((254u << 23) - __float_as_uint(s)) : 0.f;
    if (fine && (__float_as_uint(s) & 0x7fffffu)) inv = 1.0f / s;
    if (off0 && fine && s != old) {                 // the page's older codes follow the scale
      const float g = old * inv;
      for (int q = threadIdx.x; q < off0 * (D / 8); q += THREADS) {
        uint2* c = reinterpret_cast<uint2*>(pl) + q;
        uint2 w = *c;
        const float2 a0 = e4m3x2_to_f32(w.x), a1 = e4m3x2_to_f32(w.x >> 16), a2 = e4m3x2_to_f32(w.y), a3 = e4m3x2_to_f32(w.y >> 16);
        w.x = pack_e4m3x4(make_float2(a0.x * g, a0.y * g), make_float2(a1.x * g, a1.y * g));
        w.y = pack_e4m3x4(make_float2(a2.x * g, a2.y * g), make_float2(a3.x * g, a3.y * g));
        *c = w;
      }
    }
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const int r = row + i * ROWS;
      if (r < cnt) {
        uint8_t* cr = pl + (off0 + r) * D;
        if constexpr (VEC) {
          const float2 ii = make_float2(inv, inv);
          uint32_t w[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const float* a = f[i] + 4 * q;
            w[q] = pack_e4m3x4(__fmul2_rn(make_float2(a[0], a[1]), ii), __fmul2_rn(make_float2(a[2], a[3]), ii));
          }
          if (!fine) w[0] = w[1] = w[2] = w[3] = 0;
#pragma unroll
          for (int v = 0; v < R::PER; ++v) {
            uint8_t* to = cr + v * (N * TPR) + N * u;
            if constexpr (N == 8) *reinterpret_cast<uint2*>(to) = make_uint2(w[2 * v], w[2 * v + 1]);
            else *reinterpret_cast<uint32_t*>(to) = w[v];
          }
        } else {
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const int2 e = is_v ? make_int2(16 * u + 2 * k, 16 * u + 2 * k + 1) : pair_elems(tab, 8 * u + k);
            const uint32_t w = fine ? pack_e4m3x2(f[i][2 * k] * inv, f[i][2 * k + 1] * inv) : 0u;
            cr[e.x] = static_cast<uint8_t>(w);
            cr[e.y] = static_cast<uint8_t>(w >> 8);
          }
        }
      }
    }
    if (threadIdx.x == 0) *sc = s;
  }
}

template <typename T, int D, int PAGE>
cudaError_t launch(CacheAppendParams p, const RotaryTable& tab, int num_sms, cudaStream_t st) {
  auto ok16 = [](const void* q, long long a, long long b) {
    return reinterpret_cast<uintptr_t>(q) % 16 == 0 && a * sizeof(T) % 16 == 0 && b * sizeof(T) % 16 == 0;
  };
  const bool vec = (!tab.half || 2 * tab.n == D) && ok16(p.k, p.k_st, p.k_sh) && ok16(p.v, p.v_st, p.v_sh);
  p.pages_per_seq = (p.max_new + PAGE - 1) / PAGE + 1;
  const long long gx = static_cast<long long>(p.batch) * p.pages_per_seq;
  if (gx > 0x7fffffffLL) return cudaErrorInvalidValue;
  // Heads a CTA, which share the sines and hide each other's loads: as many as leave two
  // CTAs for every SM.
  const int groups = static_cast<int>(std::min<long long>(p.heads, (2LL * num_sms + 2 * gx - 1) / (2 * gx)));
  p.heads_per_cta = (p.heads + groups - 1) / groups;
  dim3 grid(static_cast<unsigned>(gx), ceil_div_i(p.heads, p.heads_per_cta), 2);
  using R = Ring<T, D, PAGE>;
  if (!vec) {
    k_cache_append<T, D, PAGE, false, false><<<grid, R::THREADS, 0, st>>>(p, tab);
    return cudaGetLastError();
  }
  // As much of the ring as the CTA's heads fill.
  const int smem = R::STAGE * std::min(R::STAGES, p.heads_per_cta);
  auto kern = tab.half ? k_cache_append<T, D, PAGE, true, true> : k_cache_append<T, D, PAGE, true, false>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, R::STAGE * R::STAGES);
  if (e != cudaSuccess) return e;
  kern<<<grid, R::THREADS, smem, st>>>(p, tab);
  return cudaGetLastError();
}

template <typename T, int D>
cudaError_t by_page(const CacheAppendParams& p, const RotaryTable& tab, int num_sms, cudaStream_t st) {
  switch (p.page_tokens) {
    case 32: return launch<T, D, 32>(p, tab, num_sms, st);
    case 64: return launch<T, D, 64>(p, tab, num_sms, st);
    default: return launch<T, D, 128>(p, tab, num_sms, st);
  }
}

template <typename T>
cudaError_t by_dim(const CacheAppendParams& p, const RotaryTable& tab, int num_sms, cudaStream_t st) {
  return p.d == 64 ? by_page<T, 64>(p, tab, num_sms, st) : by_page<T, 128>(p, tab, num_sms, st);
}

}  // namespace

cudaError_t launch_cache_append(int dtype, const CacheAppendParams& p, const RotaryTable& tab, int num_sms,
                                cudaStream_t st) {
  switch (dtype) {
    case LA_BF16: return by_dim<__nv_bfloat16>(p, tab, num_sms, st);
    case LA_FP16: return by_dim<__half>(p, tab, num_sms, st);
    default: return by_dim<float>(p, tab, num_sms, st);
  }
}
