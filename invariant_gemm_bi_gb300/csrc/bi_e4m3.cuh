// bi_e4m3.cuh -- numbers of 4 exponent and 3 mantissa bits with a scale: the
// scale of a block, rounding to e4m3 and back.
//
// The scale is 2^e, e the least integer (from -126 on) with 448 2^e at least
// the block's largest magnitude, 448 being the largest e4m3 number.  A floating
// format's rounding is relative, so a scale that uses the range up to its last
// binade gains nothing over a power of two but a binade at the small end, and a
// power of two makes scaling exact both ways: an element is rounded once.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

namespace bi {

// The scale of a block from the bits of its largest magnitude; 1 for a block of
// zeros, a NaN for one that holds a NaN or an infinity.
__device__ __forceinline__ float block_scale(uint32_t amax_bits) {
  if (amax_bits >= 0x7f800000u) return __uint_as_float(0x7fffffffu);
  if (amax_bits == 0) return 1.0f;
  // 448 = 1.75 * 2^8: the exponent of amax less 8, one more above 1.75
  const int e = (int)(amax_bits >> 23) - 127 - 8 + ((amax_bits & 0x7fffffu) > 0x600000u ? 1 : 0);
  return __uint_as_float((uint32_t)(max(e, -126) + 127) << 23);
}
// 1 / scale of a scale from block_scale, exactly: its exponent negated.
__device__ __forceinline__ float inverse_scale(float scale) {
  return scale == scale ? __uint_as_float(0x7f000000u - __float_as_uint(scale)) : scale;
}

// Two numbers rounded to e4m3 (to nearest, ties to even, at most 448; a NaN stays one), the first in the low byte.
__device__ __forceinline__ uint32_t to_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t to_e4m3x4(float a, float b, float c, float d) {
  return to_e4m3x2(a, b) | to_e4m3x2(c, d) << 16;
}
// The two pairs of four e4m3 numbers as fp16.
__device__ __forceinline__ void e4m3x4_to_half2s(uint32_t v, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 l, h;\n\t"
      "mov.b32 {l, h}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, l;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(v));
}
// Two e4m3 numbers as fp16, which holds them all.
__device__ __forceinline__ uint32_t e4m3x2_to_half2(uint32_t v) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)v));
  return r;
}
__device__ __forceinline__ float2 e4m3x2_to_float2(uint32_t v) {
  const uint32_t h = e4m3x2_to_half2(v);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

}  // namespace bi
