// la_op_rope_axes: rotation of [tokens, heads, d] by positions on several axes.
//
//   y0 = x0 cos a - x1 sin a,  y1 = x0 sin a + x1 cos a,  a = pos[t][axis] * omega
//
// (the inverse, which is also the gradient, turns by -a).  Bound: HBM, every
// element read and written once.  A thread owns one run of pairs of one token and
// walks over heads, so a sine and cosine pair is computed once for all the heads
// that the thread visits.
#include "kernels.h"
#include "rotary.cuh"

namespace {

// VEC: 16-byte accesses.  Pairs a thread owns: interleaved, the N/2 pairs of one
// 16-byte vector; halves, the N pairs of the vectors at j and n + j; passed-through
// elements, N/2 "pairs" of one vector.  Not VEC: one pair.
template <typename T, bool VEC>
__global__ void __launch_bounds__(256)
k_rope_axes(const __grid_constant__ RopeAxesParams p, const __grid_constant__ RotaryTable tab) {
  constexpr int N = Vec16<T>::N;
  const int units = p.units;
  const long long i = blockIdx.x * 256LL + threadIdx.x;
  const long long t = i / units;
  if (t >= p.tokens) return;
  const int u = static_cast<int>(i - t * units);
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
    if (tab.half) {
      float2 cs[N];
#pragma unroll
      for (int k = 0; k < N; ++k) cs[k] = pair_cos_sin(tab, u * N + k, pos);
#pragma unroll 2
      for (int h = h0; h < h1; ++h) {
        float a[N], b[N];
        Vec16<T>::unpack(*reinterpret_cast<const uint4*>(x + h * p.x_sh + u * N), a);
        Vec16<T>::unpack(*reinterpret_cast<const uint4*>(x + h * p.x_sh + tab.n + u * N), b);
#pragma unroll
        for (int k = 0; k < N; ++k) {
          const float v = a[k];
          a[k] = v * cs[k].x - b[k] * cs[k].y;
          b[k] = v * cs[k].y + b[k] * cs[k].x;
        }
        *reinterpret_cast<uint4*>(y + h * p.o_sh + u * N) = Vec16<T>::pack(a);
        *reinterpret_cast<uint4*>(y + h * p.o_sh + tab.n + u * N) = Vec16<T>::pack(b);
      }
    } else {
      float2 cs[N / 2];
#pragma unroll
      for (int k = 0; k < N / 2; ++k) cs[k] = pair_cos_sin(tab, u * (N / 2) + k, pos);
#pragma unroll 4
      for (int h = h0; h < h1; ++h) {
        float a[N];
        Vec16<T>::unpack(*reinterpret_cast<const uint4*>(x + h * p.x_sh + u * N), a);
#pragma unroll
        for (int k = 0; k < N / 2; ++k) {
          const float v = a[2 * k], w = a[2 * k + 1];
          a[2 * k] = v * cs[k].x - w * cs[k].y;
          a[2 * k + 1] = v * cs[k].y + w * cs[k].x;
        }
        *reinterpret_cast<uint4*>(y + h * p.o_sh + u * N) = Vec16<T>::pack(a);
      }
    }
  } else {
    const int2 e = pair_elems(tab, u);
    const bool turn = u < tab.n;
    const bool two = e.y < p.d;                 // an odd d passes one last element through
    const float2 cs = turn ? pair_cos_sin(tab, u, pos) : make_float2(1.f, 0.f);
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
  // Few heads a thread until the grid fills the GPU twice over, then up to 8.
  long long hpt = per_head * p.heads / (num_sms * 4096LL);
  p.heads_per_thread = static_cast<int>(hpt < 1 ? 1 : (hpt > 8 ? 8 : hpt));
  const long long gx = (per_head + 255) / 256;
  if (gx > 0x7fffffffLL) return cudaErrorInvalidValue;
  dim3 grid(static_cast<unsigned>(gx), ceil_div_i(p.heads, p.heads_per_thread));
  if (vec) k_rope_axes<T, true><<<grid, 256, 0, st>>>(p, tab);
  else k_rope_axes<T, false><<<grid, 256, 0, st>>>(p, tab);
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
