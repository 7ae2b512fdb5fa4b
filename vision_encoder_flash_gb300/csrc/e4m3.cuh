// e4m3.cuh -- 8-bit floating point, 4 exponent and 3 mantissa bits (bias 7,
// largest value 448, 0x7f and 0xff NaN, no infinities), two values at a time.
#pragma once

#include <cstdint>

namespace vattn {

// Two f32 rounded to nearest even, the first in the low byte; NaN stays NaN,
// what is beyond 448 becomes 448.
__device__ __forceinline__ uint32_t e4m3_pack(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
// Four of them, the first in the low byte.
__device__ __forceinline__ uint32_t e4m3_pack4(float a, float b, float c, float d) {
  return e4m3_pack(a, b) | e4m3_pack(c, d) << 16;
}
// The low (high) two bytes of x as a pair of f16, exactly.
__device__ __forceinline__ uint32_t e4m3_half2_lo(uint32_t x) {
  uint32_t r;
  asm("{.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;}" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ uint32_t e4m3_half2_hi(uint32_t x) {
  uint32_t r;
  asm("{.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;}" : "=r"(r) : "r"(x));
  return r;
}

// Exponent of the smallest power of two s with most <= 448 s: 448 = 1.75 * 2^8,
// so that of most less 8, and one more where its mantissa is above 1.75.
__device__ __forceinline__ int e4m3_scale_exponent(float most) {
  return static_cast<int>((__float_as_uint(most) + 0x1fffffu) >> 23) - 127 - 8;
}

}  // namespace vattn
