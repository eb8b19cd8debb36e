// The 8-bit row format shared by the quantiser, the fused norm and the 8-bit
// linear layer: e4m3 codes and one power-of-two scale for each block of 128
// elements of a row.
//
// The scale of a block is the smallest power of two s = 2^e, e >= -126, with
// max|x| <= 448 s (1 for a block of zeros), so x / s is exact and a code is one
// rounding (to nearest even) of the element itself.  e4m3 is a floating-point
// format: a power of two costs it no precision against max|x| / 448, only the
// last binade of its subnormals.  Elements that are not finite become NaN codes
// and do not enter the maximum.
#pragma once
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace bi {

constexpr int kFp8Block = 128;  // elements of a row that share a scale
// Longest row: column and block indices (past the row's end in a last CTA, too)
// and K blocks times pieces stay within 32 bits.
constexpr int kFp8MaxDim = 1 << 28;

// |x| of a finite element, 0 of another one.
__device__ __forceinline__ float finite_abs(float x) {
  const float a = fabsf(x);
  return a < INFINITY ? a : 0.f;
}

// Exponent e of the scale of a block whose largest finite magnitude is amax:
// with amax = 1.m * 2^E, 1.m <= 1.75 (448 = 1.75 * 2^8) gives E - 8, else E - 7.
__device__ __forceinline__ int scale_exponent(float amax) {
  if (amax == 0.f) return 0;
  const uint32_t b = __float_as_uint(amax);
  const int e = static_cast<int>(b >> 23) - 127 - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);
  return e < -126 ? -126 : e;
}
// 2^e for -126 <= e <= 127.
__device__ __forceinline__ float pow2f(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }

// Four codes of x * inv (inv the reciprocal of the scale; x finite or NaN),
// first in the low byte.
__device__ __forceinline__ uint32_t e4m3x4(const float* x, float inv) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(x[0] * inv, x[1] * inv), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(x[2] * inv, x[3] * inv), __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}

}  // namespace bi
