// la_op_rope_axes: rotation of [tokens, heads, d] by positions on several axes.
//
//   y0 = x0 cos a - x1 sin a,  y1 = x0 sin a + x1 cos a,  a = pos[t][axis] * omega
//
// (the inverse, which is also the gradient, turns by -a).  Bound: HBM, every
// element read and written once.  A thread owns one run of pairs of one token and
// walks over heads, so a sine and cosine pair is computed once for all the heads
// that the thread visits; it reads BATCH heads before it writes the first of them,
// which keeps that many 16-byte loads under way (in place, too: the elements are its
// own).
#include "kernels.h"
#include "rotary.cuh"

namespace {

constexpr int BATCH = 4;

// VEC: 16-byte accesses (HALF: tab.half).  Pairs a thread owns: interleaved, the N/2 pairs of one
// 16-byte vector; halves, the N pairs of the vectors at j and n + j; passed-through
// elements, N/2 "pairs" of one vector.  Not VEC: one pair.
template <typename T, bool VEC, bool HALF>
__global__ void __launch_bounds__(256)
k_rope_axes(const __grid_constant__ RopeAxesParams p, const __grid_constant__ RotaryTable tab) {
  constexpr int N = Vec16<T>::N;
  __shared__ PairTable pairs;
  pairs.fill(tab);
  __syncthreads();
  // A CTA's 256 units start at token t0, unit u0 of it.
  const long long i0 = blockIdx.x * 256LL;
  const long long t0 = i0 / p.units;
  const unsigned at = static_cast<unsigned>(i0 - t0 * p.units) + threadIdx.x;
  const long long t = t0 + at / static_cast<unsigned>(p.units);
  if (t >= p.tokens) return;
  const int u = static_cast<int>(at % static_cast<unsigned>(p.units));
  const int h0 = blockIdx.y * p.heads_per_thread;
  const int h1 = min(h0 + p.heads_per_thread, p.heads);
  const int* pos = p.pos + t * tab.naxes;
  const T* x = static_cast<const T*>(p.x) + t * p.x_st;
  T* y = static_cast<T*>(p.out) + t * p.o_st;
  if constexpr (VEC) {
    const int rot_units = tab.half ? tab.n / N : 2 * tab.n / N;
    if (u >= rot_units) {                       // passed through
      const int e = 2 * tab.n + (u - rot_units) * N;
      for (int h = h0; h < h1; ++h)
        *reinterpret_cast<uint4*>(y + h * p.o_sh + e) = *reinterpret_cast<const uint4*>(x + h * p.x_sh + e);
      return;
    }
    const int lo = u * N, hi = tab.half ? tab.n + u * N : 0;
    float2 cs[N];
    for (int h = h0; h < h1; h += BATCH) {
      uint4 a[BATCH], b[BATCH];
#pragma unroll
      for (int k = 0; k < BATCH; ++k) {
        if (h + k >= h1) continue;
        a[k] = *reinterpret_cast<const uint4*>(x + (h + k) * p.x_sh + lo);
        if (HALF) b[k] = *reinterpret_cast<const uint4*>(x + (h + k) * p.x_sh + hi);
      }
      if (h == h0) {                            // behind the first loads
#pragma unroll
        for (int k = 0; k < (HALF ? N : N / 2); ++k) cs[k] = pairs.cos_sin(u * (HALF ? N : N / 2) + k, pos, tab.inverse);
      }
#pragma unroll
      for (int k = 0; k < BATCH; ++k) {
        if (h + k >= h1) continue;
        float f[N], g[N];
        Vec16<T>::unpack(a[k], f);
        if constexpr (HALF) {
          Vec16<T>::unpack(b[k], g);
#pragma unroll
          for (int e = 0; e < N; ++e) {
            const float v = f[e];
            f[e] = v * cs[e].x - g[e] * cs[e].y;
            g[e] = v * cs[e].y + g[e] * cs[e].x;
          }
          *reinterpret_cast<uint4*>(y + (h + k) * p.o_sh + hi) = Vec16<T>::pack(g);
        } else {
#pragma unroll
          for (int e = 0; e < N / 2; ++e) {
            const float v = f[2 * e], w = f[2 * e + 1];
            f[2 * e] = v * cs[e].x - w * cs[e].y;
            f[2 * e + 1] = v * cs[e].y + w * cs[e].x;
          }
        }
        *reinterpret_cast<uint4*>(y + (h + k) * p.o_sh + lo) = Vec16<T>::pack(f);
      }
    }
  } else {
    const int2 e = pair_elems(tab, u);
    const bool turn = u < tab.n;
    const bool two = e.y < p.d;                 // an odd d passes one last element through
    const float2 cs = turn ? pairs.cos_sin(u, pos, tab.inverse) : make_float2(1.f, 0.f);
    for (int h = h0; h < h1; ++h) {
      const T* xr = x + h * p.x_sh;
      T* yr = y + h * p.o_sh;
      if (!turn) {
        const T v0 = xr[e.x];
        if (two) yr[e.y] = xr[e.y];
        yr[e.x] = v0;
        continue;
      }
      const float v = to_f32(xr[e.x]), w = to_f32(xr[e.y]);
      yr[e.x] = from_f32<T>(v * cs.x - w * cs.y);
      yr[e.y] = from_f32<T>(v * cs.y + w * cs.x);
    }
  }
}

template <typename T>
cudaError_t launch(RopeAxesParams p, const RotaryTable& tab, int num_sms, cudaStream_t st) {
  constexpr int N = Vec16<T>::N;
  auto ok16 = [](const void* q, long long a, long long b) {
    return reinterpret_cast<uintptr_t>(q) % 16 == 0 && a * sizeof(T) % 16 == 0 && b * sizeof(T) % 16 == 0;
  };
  const int rot = tab.half ? tab.n : 2 * tab.n;
  const bool vec = p.d % N == 0 && rot % N == 0 && 2 * tab.n % N == 0 && ok16(p.x, p.x_st, p.x_sh) && ok16(p.out, p.o_st, p.o_sh);
  p.units = vec ? rot / N + (p.d - 2 * tab.n) / N : (p.d + 1) / 2;
  const long long per_head = p.tokens * p.units;
  // One head a thread until the grid has 1024 threads for every SM, then up to 8: the
  // sines are shared and more loads are under way (every output in memory of its own, 4680
  // x 40 x 128 bf16: 18.1 us, 18.2 with 4096; 3601 x 24 x 64 fp32 halves: 9.9, 11.4 with
  // 2048, 15.9 with 4096).
  const long long hpt = per_head * p.heads / (num_sms * 1024LL);
  p.heads_per_thread = static_cast<int>(hpt < 1 ? 1 : (hpt > 8 ? 8 : hpt));
  const long long gx = (per_head + 255) / 256;
  if (gx > 0x7fffffffLL) return cudaErrorInvalidValue;
  dim3 grid(static_cast<unsigned>(gx), ceil_div_i(p.heads, p.heads_per_thread));
  if (!vec) k_rope_axes<T, false, false><<<grid, 256, 0, st>>>(p, tab);
  else if (tab.half) k_rope_axes<T, true, true><<<grid, 256, 0, st>>>(p, tab);
  else k_rope_axes<T, true, false><<<grid, 256, 0, st>>>(p, tab);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rope_axes(int dtype, const RopeAxesParams& p, const RotaryTable& tab, int num_sms, cudaStream_t st) {
  switch (dtype) {
    case LA_BF16: return launch<__nv_bfloat16>(p, tab, num_sms, st);
    case LA_FP16: return launch<__half>(p, tab, num_sms, st);
    default: return launch<float>(p, tab, num_sms, st);
  }
}
