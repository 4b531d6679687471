// quant.cuh -- K/V held in 8 bits: e4m3 payloads with one fp32 scale for a
// block of tokens and K/V head.
#pragma once

#include <cuda_fp8.h>

#include "common.cuh"

namespace dc {
namespace {

// Scales that the library makes are powers of two in 2^-64 .. 2^64: a raised
// scale then moves exponents only, and an older payload loses no more than what
// falls below e4m3's least step, 2^-9.
constexpr int kScaleLow = -64, kScaleHigh = 64;

// Two finite values to e4m3, to nearest even, at most 448.
__device__ __forceinline__ uint32_t finite_e4m3x2(float a, float b) {
  return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}
// Two values to e4m3, to nearest even.  Infinities become NaN like NaN itself:
// a largest finite value in their place would pass for data.
__device__ __forceinline__ uint32_t to_e4m3x2(float a, float b) {
  uint32_t r = finite_e4m3x2(a, b);
  if ((__float_as_uint(a) & 0x7F800000u) == 0x7F800000u) r |= 0x7Fu;
  if ((__float_as_uint(b) & 0x7F800000u) == 0x7F800000u) r |= 0x7F00u;
  return r;
}
__device__ __forceinline__ float2 from_e4m3x2(uint32_t x) {
  return __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)x, __NV_E4M3)));
}

// The least power of two s (within the bounds above) with most <= 448 s; most
// finite and not negative.  448 = 1.75 x 2^8.
__device__ __forceinline__ float least_scale(float most) {
  const uint32_t b = __float_as_uint(most);
  const int e = (int)(b >> 23) - 127 - ((b & 0x7FFFFFu) <= 0x600000u ? 8 : 7);
  return __uint_as_float((uint32_t)(min(max(e, kScaleLow), kScaleHigh) + 127) << 23);
}

}  // namespace
}  // namespace dc
