// E4M3 with one fp32 scale per group of 128 values, the form of activation checkpoints.
#pragma once

#include "common.cuh"

namespace moe {

constexpr int FP8_GROUP = 128;

// Largest magnitude that keeps a NaN: magnitudes order as integers, with NaN above infinity.
__device__ __forceinline__ float fp8_amax(float a, float b) {
  return __uint_as_float(max(__float_as_uint(a) & 0x7FFFFFFFu, __float_as_uint(b) & 0x7FFFFFFFu));
}

// Scale of a group whose largest magnitude is amax: the product amax * fp32(1 / 448), rounded once, by definition.  It is
// an ulp away from the quotient amax / 448 in about half of all groups; the codes are of x over the scale as it came out, so
// neither is the nearer one to x.  1 where the product is zero, NaN for a group with a NaN or an infinity (its codes are 0).
__device__ __forceinline__ float fp8_scale(float amax) {
  if (!(amax < __uint_as_float(0x7F800000u))) return __uint_as_float(0x7FC00000u);
  const float s = __fmul_rn(amax, 1.0f / 448.0f);
  return s > 0.0f ? s : 1.0f;
}

// Two codes, the first in the low byte: to nearest with ties to even, saturating at 448.
__device__ __forceinline__ uint32_t fp8_pair(float a, float b) {
  return (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}

// The values of the two codes in the low half of c.
__device__ __forceinline__ float2 fp8_unpair(uint32_t c) {
  return __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)c, __NV_E4M3)));
}

}  // namespace moe
