// sa_e4m3.cuh — e4m3 codes (sign, four exponent bits, three of the mantissa; 448 the largest value, 0x7F and 0xFF not
// numbers, no infinities) and the scales of a cache that holds them.
#pragma once

#include <stdint.h>

namespace sa {

// A block's scale as it counts: one that is not a positive finite number marks an empty block, whose values are 0.
__device__ __forceinline__ float held_scale(float s) { return s > 0.f && s <= 3.4028234663852886e38f ? s : 0.f; }

// The least power of two s, 2^-126 at least, with top / s <= 448 = 1.75 2^8; 0 for top = 0.  (top finite, >= 0)
__device__ __forceinline__ float scale_for(float top) {
  const uint32_t u = __float_as_uint(top);
  if (u == 0) return 0.f;
  const int e = static_cast<int>(u >> 23) - 8 + ((u & 0x7FFFFFu) > 0x600000u);
  return __uint_as_float(static_cast<uint32_t>(e < 1 ? 1 : e) << 23);
}

// Two values to the nearest codes (ties to even, past 448: 448; a NaN stays one), lo in the low byte.
__device__ __forceinline__ uint32_t encode2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// Two codes as a pair of fp16 values (exact), the low byte's in the low half.
__device__ __forceinline__ uint32_t decode2(uint32_t codes) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(codes)));
  return r;
}

__device__ __forceinline__ float half_lo(uint32_t pair) {
  float r;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.f32.f16 %0, lo;\n\t}" : "=f"(r) : "r"(pair));
  return r;
}
__device__ __forceinline__ float half_hi(uint32_t pair) {
  float r;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.f32.f16 %0, hi;\n\t}" : "=f"(r) : "r"(pair));
  return r;
}

}  // namespace sa
