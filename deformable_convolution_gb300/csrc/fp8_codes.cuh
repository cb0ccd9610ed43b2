// Codes and scales of values in registers.
#pragma once

#include <cuda_fp8.h>

#include "fp8.cuh"

namespace dc {
namespace {

__device__ __forceinline__ uint32_t magnitude(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// The scale byte of a block whose largest magnitude has these bits: exponent
// e = exponent(top) - high (+ 1 where top's mantissa is above 1.75), so that
// top / 2^e is at most 1.75 * 2^high, the largest code.  Bits order like
// magnitudes, and what is not finite sorts above.
template <int FMT>
__device__ __forceinline__ uint32_t scale_byte(uint32_t top) {
  if (top >= 0x7f800000u) return 255u;
  constexpr int high = FMT == DC_E4M3 ? 8 : 15;
  const int e = (int)(top >> 23) - high + ((top & 0x7fffffu) > 0x600000u ? 1 : 0);
  return (uint32_t)(e < 1 ? 1 : e);
}

// 2^-(byte - 127): exact for bytes 1 .. 254 (those that blocks have are at
// most 247); NaN for 255, which makes the block's codes NaN.
__device__ __forceinline__ float inverse_scale(uint32_t byte) {
  return byte == 255u ? __uint_as_float(0x7fffffffu) : __uint_as_float((254u - byte) << 23);
}

// Two codes of scaled values, rounded to nearest even; `a` in the low byte.
template <int FMT>
__device__ __forceinline__ uint32_t codes2(float a, float b) {
  const __nv_fp8x2_storage_t c = __nv_cvt_float2_to_fp8x2(
      make_float2(a, b), __NV_SATFINITE, FMT == DC_E4M3 ? __NV_E4M3 : __NV_E5M2);
  return (uint32_t)c;
}

// A thread's eight consecutive values of a row.
template <typename T>
struct Eight;
template <>
struct Eight<float> {
  float v[8];
  __device__ __forceinline__ float get(int i) const { return v[i]; }
  __device__ __forceinline__ void load(const float* p) {
    const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  }
  __device__ __forceinline__ void load_some(const float* p, int count) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < count ? p[i] : 0.f;
  }
  __device__ __forceinline__ uint32_t top() const {
    uint32_t t = 0u;
#pragma unroll
    for (int i = 0; i < 8; ++i) t = max(t, magnitude(v[i]));
    return t;
  }
};
template <>
struct Eight<__nv_bfloat16> {
  uint32_t w[4];
  __device__ __forceinline__ float get(int i) const {
    return __uint_as_float(i & 1 ? w[i >> 1] & 0xffff0000u : w[i >> 1] << 16);
  }
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    const uint4 a = *reinterpret_cast<const uint4*>(p);
    w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w;
  }
  __device__ __forceinline__ void load_some(const __nv_bfloat16* p, int count) {
    const unsigned short* q = reinterpret_cast<const unsigned short*>(p);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] = (2 * i < count ? (uint32_t)q[2 * i] : 0u) | (2 * i + 1 < count ? (uint32_t)q[2 * i + 1] << 16 : 0u);
  }
  __device__ __forceinline__ uint32_t top() const {
    uint32_t t = 0u;
#pragma unroll
    for (int i = 0; i < 4; ++i) t = __vmaxu2(t, w[i] & 0x7fff7fffu);
    return max(t & 0xffff0000u, t << 16);
  }
};

// The largest magnitudes of a thread's columns over its rows.
template <typename T>
__device__ __forceinline__ void column_tops(const Eight<T>* x, uint32_t* top);
template <>
__device__ __forceinline__ void column_tops<float>(const Eight<float>* x, uint32_t* top) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    uint32_t t = 0u;
#pragma unroll
    for (int r = 0; r < 8; ++r) t = max(t, magnitude(x[r].v[i]));
    top[i] = max(t, __shfl_xor_sync(0xffffffffu, t, 16));
  }
}
template <>
__device__ __forceinline__ void column_tops<__nv_bfloat16>(const Eight<__nv_bfloat16>* x, uint32_t* top) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t t = 0u;
#pragma unroll
    for (int r = 0; r < 8; ++r) t = __vmaxu2(t, x[r].w[i] & 0x7fff7fffu);
    t = __vmaxu2(t, __shfl_xor_sync(0xffffffffu, t, 16));
    top[2 * i] = t << 16;
    top[2 * i + 1] = t & 0xffff0000u;
  }
}

}  // namespace
}  // namespace dc
