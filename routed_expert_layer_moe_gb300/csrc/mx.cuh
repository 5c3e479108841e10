// MXFP4 on the device: blocks of 32 values that share one power-of-two scale (OCP
// Microscaling Formats v1.0, conversion rule of section 6.3 with E2M1 elements).
#pragma once

#include <cuda_fp4.h>

#include "common.cuh"

namespace moe {

constexpr int MX_BLOCK = 32;

// Scale byte of a block whose largest magnitude is amax: e = floor(log2 amax) - 2 (2 = the
// exponent of E2M1's largest binade, 4..6), clamped to [-127, 125], biased by 127; 127 for an
// all-zero block and 255 for one with a NaN or an infinity.  The exponent field of a subnormal
// amax is 0, whose e = -129 the clamp lifts to -127, as it does the subnormal's true exponent.
__device__ __forceinline__ uint32_t mx_scale_byte(float amax) {
  const uint32_t bits = __float_as_uint(amax);
  const int f = (int)((bits >> 23) & 0xFFu);
  if (f == 255) return 255u;
  if (bits == 0u) return 127u;
  return (uint32_t)max(f - 2, 0);
}

// 2^-(s - 127): the factor of a block's values before rounding (0 for s = 255, whose codes are
// 0).  2^127 for s = 0 down to 2^-125 for s = 252: always a normal number.
__device__ __forceinline__ float mx_inv_scale(uint32_t s) {
  return s == 255u ? 0.0f : __uint_as_float((254u - s) << 23);
}

// 2^(s - 127), a subnormal number for s = 0, NaN for s = 255.
__device__ __forceinline__ float mx_scale(uint32_t s) {
  if (s == 255u) return __uint_as_float(0x7FC00000u);
  return __uint_as_float(s ? s << 23 : 0x00400000u);
}

// Largest magnitude that keeps a NaN: the bit patterns of magnitudes order as integers, with
// NaN above infinity.
__device__ __forceinline__ float mx_amax(float a, float b) {
  return __uint_as_float(max(__float_as_uint(a) & 0x7FFFFFFFu, __float_as_uint(b) & 0x7FFFFFFFu));
}

// max(|a|, |b|, |c|), NaN if one of them is.
__device__ __forceinline__ float mx_amax3(float a, float b, float c) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// Eight codes (4 bytes) of v[0..7] * inv, the first in the lowest nibble (nearest, ties to even,
// saturating).  inv = 0 (a block with a NaN or an infinity): zeros.
__device__ __forceinline__ uint32_t mx_codes8(const float* v, float inv) {
  const float2 s = make_float2(inv, inv);
  float2 a[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) a[i] = __fmul2_rn(make_float2(v[2 * i], v[2 * i + 1]), s);
  uint32_t r;
  asm("{\n"
      "  .reg .b8 b0, b1, b2, b3;\n"
      "  cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n"
      "  cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n"
      "  cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n"
      "  cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n"
      "  mov.b32 %0, {b0, b1, b2, b3};\n"
      "}\n"
      : "=r"(r)
      : "f"(a[0].x), "f"(a[0].y), "f"(a[1].x), "f"(a[1].y), "f"(a[2].x), "f"(a[2].y), "f"(a[3].x), "f"(a[3].y));
  return inv == 0.0f ? 0u : r;
}

}  // namespace moe
