// E4M3 codes under a power-of-two scale, shared by the norm's MXFP8 output, the 8-bit cache
// and the products that read MXFP8.
//
// The scale of a set of values is the smallest X = 2^e with max |v| <= 448 X (448 = 1.75 2^8,
// the largest E4M3 value): with max |v| = f 2^k, 1 <= f < 2, e = k - 8, or k - 7 where f > 1.75.
// No finite value saturates, and scaling by 2^-e is exact, so a code is v rounded once.
#pragma once

#include <cstdint>

#include "lc_common.cuh"

namespace lc {

// |v| where it is finite, else 0: what takes part in the maximum of a set
__device__ __forceinline__ float finite_abs(float v) {
  const float a = fabsf(v);
  return a < INFINITY ? a : 0.f;  // false for NaN too
}

// e for a maximum amax > 0 (finite); subnormal maxima get an exponent below any clamp in use
__device__ __forceinline__ int e4m3_scale_exp(float amax) {
  const uint32_t u = __float_as_uint(amax);
  return static_cast<int>(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
}

// 2^e for -126 <= e <= 127
__device__ __forceinline__ float pow2f(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }

// four values -> four E4M3 bytes (round to nearest even, saturating), little-endian
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  return static_cast<uint32_t>(f32x2_to_e4m3x2(a, b)) | (static_cast<uint32_t>(f32x2_to_e4m3x2(c, d)) << 16);
}

}  // namespace lc
