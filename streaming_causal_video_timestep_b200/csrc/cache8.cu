// la_op_cache_append_fp8: new keys (rotated on the way) and values into pages of
// e4m3 codes with one power-of-two scale for each (page, head).
//
// One CTA takes one page of one sequence, for K or for V, and walks over heads:
// it holds the page's new tokens in registers (fp32, after the rotation), reduces
// their largest magnitude over the CTA, picks the scale and writes the codes, so
// every new element is read once and every code written once.  Bound: HBM.
//
// Scale: 2^k, the smallest with 448 * 2^k >= amax (k >= -64), read off amax's own
// exponent and mantissa, so no rounding decides it.  A page that already holds
// tokens keeps the larger of its scale and that; where it grows, the codes in
// front of the new tokens are multiplied by old / new, a power of two, and rounded
// to e4m3 again: exact but for results below e4m3's normal range.  A magnitude
// that is not finite makes the scale NaN, which marks the page's head until its
// first token is written again.
#include "kernels.h"
#include "rotary.cuh"
#include "sm100.cuh"

namespace {

constexpr int THREADS = 256;

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

// A thread owns 8 pairs of one token a pass: pairs 8u .. 8u+7 of its row, D/16
// threads a row.  VEC: the pairs' elements are 16-byte vectors of the input and 16
// (or twice 8) consecutive codes.
template <typename T, int D, int PAGE, bool VEC>
__global__ void __launch_bounds__(THREADS)
k_cache_append(const __grid_constant__ CacheAppendParams p, const __grid_constant__ RotaryTable tab) {
  constexpr int TPR = D / 16;                       // threads a row
  constexpr int ROWS = THREADS / TPR;               // rows a pass
  constexpr int NP = (PAGE + ROWS - 1) / ROWS;
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

  float2 cs[NP][8];
  const bool rotate = !is_v && tab.n > 0;
  if (rotate) {
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const int r = row + i * ROWS;
#pragma unroll
      for (int k = 0; k < 8; ++k)
        cs[i][k] = r < cnt && 8 * u + k < tab.n ? pair_cos_sin(tab, 8 * u + k, p.pos + (tok0 + r) * tab.naxes) : make_float2(1.f, 0.f);
    }
  }
  __shared__ uint32_t red[2][THREADS / 32];
  const int h0 = blockIdx.y * p.heads_per_cta, h1 = min(h0 + p.heads_per_cta, p.heads);
  const T* x = static_cast<const T*>(is_v ? p.v : p.k);
  const long long st = is_v ? p.v_st : p.k_st, sh = is_v ? p.v_sh : p.k_sh;
  float* scales = is_v ? p.v_scale : p.k_scale;
  uint8_t* pages = is_v ? p.v_pages : p.k_pages;
  const bool half = tab.half && !is_v && 8 * u < tab.n;   // this thread's pairs lie n apart

  for (int h = h0; h < h1; ++h) {
    float f[NP][16];                                // pair k of the 8: f[2k], f[2k+1]
    uint32_t amax = 0;
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const int r = row + i * ROWS;
      if (r < cnt) {
        const T* xr = x + (tok0 + r) * st + h * sh;
        if constexpr (VEC) {
          float a[16];
          const T* lo = half ? xr + 8 * u : xr + 16 * u;
          const T* hi = half ? xr + tab.n + 8 * u : xr + 16 * u + 8;
#pragma unroll
          for (int w = 0; w < 8 / N; ++w) {
            Vec16<T>::unpack(*reinterpret_cast<const uint4*>(lo + w * N), a + w * N);
            Vec16<T>::unpack(*reinterpret_cast<const uint4*>(hi + w * N), a + 8 + w * N);
          }
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            f[i][2 * k] = half ? a[k] : a[2 * k];
            f[i][2 * k + 1] = half ? a[8 + k] : a[2 * k + 1];
          }
        } else {
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
            if (8 * u + k < tab.n) {
              const float v = f[i][2 * k], w = f[i][2 * k + 1];
              f[i][2 * k] = v * cs[i][k].x - w * cs[i][k].y;
              f[i][2 * k + 1] = v * cs[i][k].y + w * cs[i][k].x;
            }
          }
        }
#pragma unroll
        for (int k = 0; k < 16; ++k) amax = max(amax, __float_as_uint(f[i][k]) & 0x7fffffffu);   // NaN > inf > finite
      } else {
#pragma unroll
        for (int k = 0; k < 16; ++k) f[i][k] = 0.f;
      }
    }
    amax = __reduce_max_sync(0xffffffffu, amax);
    uint32_t* rd = red[(h - h0) & 1];
    if (threadIdx.x % 32 == 0) rd[threadIdx.x / 32] = amax;
    float* sc = scales + static_cast<long long>(pg) * p.heads + h;
    const float old = off0 ? *sc : 0.f;             // read by every thread before thread 0 writes it
    __syncthreads();
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) amax = max(amax, rd[w]);
    float s = page_scale(amax);
    if (off0) s = (old != old || s != s) ? __uint_as_float(0x7fc00000u) : fmaxf(old, s);
    const bool fine = s == s;
    const float inv = fine ? 1.0f / s : 0.f;        // a power of two: exact
    uint8_t* pl = pages + (static_cast<long long>(pg) * p.heads + h) * (PAGE * D);
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
        if (!fine) {
#pragma unroll
          for (int k = 0; k < 16; ++k) f[i][k] = 0.f;
        }
        if constexpr (VEC) {
          float a[16];
#pragma unroll
          for (int k = 0; k < 16; ++k) a[k] = (half ? f[i][k < 8 ? 2 * k : 2 * k - 15] : f[i][k]) * inv;
          uint32_t w[4];
#pragma unroll
          for (int q = 0; q < 4; ++q)
            w[q] = pack_e4m3x4(make_float2(a[4 * q], a[4 * q + 1]), make_float2(a[4 * q + 2], a[4 * q + 3]));
          if (half) {
            *reinterpret_cast<uint2*>(cr + 8 * u) = make_uint2(w[0], w[1]);
            *reinterpret_cast<uint2*>(cr + tab.n + 8 * u) = make_uint2(w[2], w[3]);
          } else {
            *reinterpret_cast<uint4*>(cr + 16 * u) = make_uint4(w[0], w[1], w[2], w[3]);
          }
        } else {
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const int2 e = is_v ? make_int2(16 * u + 2 * k, 16 * u + 2 * k + 1) : pair_elems(tab, 8 * u + k);
            const uint32_t w = pack_e4m3x2(f[i][2 * k] * inv, f[i][2 * k + 1] * inv);
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
  // Halves: a thread's 8 pairs are either all rotated or all passed through.
  const bool vec = (!tab.half || tab.n % 8 == 0) && ok16(p.k, p.k_st, p.k_sh) && ok16(p.v, p.v_st, p.v_sh);
  p.pages_per_seq = (p.max_new + PAGE - 1) / PAGE + 1;
  const long long gx = static_cast<long long>(p.batch) * p.pages_per_seq;
  if (gx > 0x7fffffffLL) return cudaErrorInvalidValue;
  // Heads a CTA, which share the sines: one until the grid fills the GPU, then up to 8.
  long long hpc = gx * 2 * p.heads / (num_sms * 4LL);
  p.heads_per_cta = static_cast<int>(hpc < 1 ? 1 : (hpc > 8 ? 8 : hpc));
  dim3 grid(static_cast<unsigned>(gx), ceil_div_i(p.heads, p.heads_per_cta), 2);
  if (vec) k_cache_append<T, D, PAGE, true><<<grid, THREADS, 0, st>>>(p, tab);
  else k_cache_append<T, D, PAGE, false><<<grid, THREADS, 0, st>>>(p, tab);
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
