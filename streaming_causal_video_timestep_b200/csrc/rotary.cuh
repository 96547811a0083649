// Rotary positions with several axes, shared by k_rope_axes and the cache append.
//
// Pair j (of n) turns by pos[axis(j)] * omega_j.  The angle is kept in turns as a
// 64-bit fixed-point fraction: omega_j / (2 pi) * 2^64 comes from the host, 2^-60 turns
// off at most, and the product with the (signed) position wraps modulo 2^64, which is
// exactly "modulo one turn".  Its error is |pos| * 2^-60 turns at most, for every position
// an int32 holds, where pos * omega in fp32 would lose 2^-24 * pos * omega radians (6e-3
// at position 1e5).  Its top 32 bits, as an integer, give the quadrant and the signed
// rest within an eighth of a turn exactly; the rest goes to fp32 once and into the
// Taylor series of sine and cosine about 0 (next terms at pi/4: 3e-9 and 4e-10).
#pragma once

#include <cuda_fp16.h>

#include "kernels.h"

// Elements of pair j of a row: the rotated pairs first, then the elements that
// pass through, two by two (j >= n in either layout).
__device__ __forceinline__ int2 pair_elems(const RotaryTable& t, int j) {
  if (t.half && j < t.n) return make_int2(j, j + t.n);
  return make_int2(2 * j, 2 * j + 1);
}

__device__ __forceinline__ float2 turn_cos_sin(uint32_t turn) {   // turn: of 2^32
  const uint32_t q = (turn + 0x20000000u) >> 30;
  const float u = static_cast<float>(static_cast<int>(turn - (q << 30))) * 1.4629180792671596e-9f;   // 2 pi / 2^32
  const float w = u * u;
  float s = fmaf(w, 2.7557319223985893e-6f, -1.9841269841269841e-4f);   // 1/9!, -1/7!
  s = fmaf(s, w, 8.3333333333333333e-3f);                                // 1/5!
  s = fmaf(s, w, -1.6666666666666667e-1f);                               // -1/3!
  s = fmaf(s * w, u, u);
  float c = fmaf(w, -2.7557319223985888e-7f, 2.4801587301587302e-5f);   // -1/10!, 1/8!
  c = fmaf(c, w, -1.3888888888888889e-3f);                               // -1/6!
  c = fmaf(c, w, 4.1666666666666664e-2f);                                // 1/4!
  c = fmaf(c, w, -0.5f);
  c = fmaf(c, w, 1.0f);
  const float a = q & 1 ? s : c, b = q & 1 ? c : s;                      // |cos|, |sin| up to their signs
  return make_float2((q + 1) & 2 ? -a : a, q & 2 ? -b : b);
}

// The table's pairs in shared memory: lanes of a warp ask for different pairs, which the
// constant bank that holds the launch's arguments would serve one after the other.
// Filled by all threads of the CTA; they meet before they use it.
struct PairTable {
  unsigned long long turn[LA_ROPE_MAX_PAIRS];
  unsigned char axis[LA_ROPE_MAX_PAIRS];
  __device__ __forceinline__ void fill(const RotaryTable& t) {
    for (int j = threadIdx.x; j < t.n; j += blockDim.x) {
      turn[j] = t.turn[j];
      axis[j] = t.axis[j];
    }
  }
  __device__ __forceinline__ float2 cos_sin(int j, const int* pos, bool inverse) const {
    const unsigned long long ph = static_cast<unsigned long long>(static_cast<long long>(pos[axis[j]])) * turn[j];
    const float2 v = turn_cos_sin(static_cast<uint32_t>(ph >> 32));
    return make_float2(v.x, inverse ? -v.y : v.y);
  }
  // The same, each the fp32 value nearest to that of the table's angle (computed in fp64),
  // and so of the exact one but where |pos| * 2^-60 turns decide.
  __device__ __forceinline__ float2 cos_sin_nearest(int j, const int* pos) const {
    const unsigned long long ph = static_cast<unsigned long long>(static_cast<long long>(pos[axis[j]])) * turn[j];
    double s, c;
    sincospi(static_cast<double>(static_cast<long long>(ph)) * 1.0842021724855044e-19 /* 2^-63 */, &s, &c);
    return make_float2(static_cast<float>(c), static_cast<float>(s));
  }
};

template <typename T> struct Vec16;             // 16 bytes of T as fp32 values
template <> struct Vec16<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ void unpack(uint4 u, float* f) {
    f[0] = __uint_as_float(u.x); f[1] = __uint_as_float(u.y); f[2] = __uint_as_float(u.z); f[3] = __uint_as_float(u.w);
  }
  static __device__ __forceinline__ uint4 pack(const float* f) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
  }
};
template <> struct Vec16<__nv_bfloat16> {
  static constexpr int N = 8;
  static __device__ __forceinline__ void unpack(uint4 u, float* f) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ uint4 pack(const float* f) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      __nv_bfloat162 v = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      w[i] = *reinterpret_cast<uint32_t*>(&v);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};
template <> struct Vec16<__half> {
  static constexpr int N = 8;
  static __device__ __forceinline__ void unpack(uint4 u, float* f) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      f[2 * i] = v.x;
      f[2 * i + 1] = v.y;
    }
  }
  static __device__ __forceinline__ uint4 pack(const float* f) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      __half2 v = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
      w[i] = *reinterpret_cast<uint32_t*>(&v);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
template <typename T> __device__ __forceinline__ T from_f32(float v);
template <> __device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <> __device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }
