// The quantised cache's number format, on the device: 8-bit floats of four
// significant bits (e4m3) with one power of two for the head of a token.
//
// The scale is 2^(byte - 127) with the smallest byte >= 1 that brings the largest
// finite value of the head to 448 or less, the largest code. Codes are floating
// point themselves, so a scale nearer to max / 448 would give no value more
// precision, only half an octave of the seventeen that a head's codes span; and
// with a power of two scaling never rounds, so a cached value is rounded once, and
// a cached bf16 value of four significant bits not at all.
#pragma once

#include "common.hpp"

namespace sc {

// Two codes of a word as bf16 values, times a power of two: for every code and byte the
// product rounded once to bf16, subnormal and infinite ones too.
__device__ __forceinline__ uint32_t fp8_pair_lo(uint32_t w, float by = 1.f) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, by, false));
}
__device__ __forceinline__ uint32_t fp8_pair_hi(uint32_t w, float by = 1.f) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, by, true));
}

// Eight codes (two words) as eight bf16 values, times a power of two.
__device__ __forceinline__ u32x4 fp8_to_bf16(uint32_t w0, uint32_t w1, float by = 1.f) {
  return u32x4{fp8_pair_lo(w0, by), fp8_pair_hi(w0, by), fp8_pair_lo(w1, by), fp8_pair_hi(w1, by)};
}

// A scale as the float whose exponent the conversions take; that of 0 counts as 2^-127.
__device__ __forceinline__ float scale_float(uint32_t byte) { return __uint_as_float(byte << 23); }

// Sixteen codes times their scale.
__device__ __forceinline__ void fp8_to_bf16_scaled(u32x4 w, uint32_t byte, u32x4* y) {
  const float by = scale_float(byte);
  y[0] = fp8_to_bf16(w[0], w[1], by);
  y[1] = fp8_to_bf16(w[2], w[3], by);
}

// The scale's byte for a head whose largest finite value has these bits (no sign):
// 448 = 1.75 2^8, so a mantissa above 1.75 takes one more.
__device__ __forceinline__ int scale_byte(uint32_t top) {
  return max((int)((top + 0x1FFFFFu) >> 23) - 8, 1);
}

// 2^(127 - byte) for a byte that scale_byte gives (1 .. 247).
__device__ __forceinline__ float scale_inverse(int byte) {
  return __uint_as_float((uint32_t)(254 - byte) << 23);
}

// Four values as codes, rounded to nearest even; what is not finite becomes NaN.
__device__ __forceinline__ uint32_t to_fp8(const float* f, float inv) {
  float y[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) y[e] = fabsf(f[e]) < INFINITY ? f[e] * inv : __uint_as_float(0x7FC00000u);
  const int w = __builtin_amdgcn_cvt_pk_fp8_f32(y[0], y[1], 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(y[2], y[3], w, true);
}

}  // namespace sc
