// fp8.cuh -- e4m3 <-> fp16/fp32 conversions and the block scales of the
// 8-bit cache.
//
// A block of rows is held as e4m3 codes and one fp32 scale 2^e, e the least
// integer with amax <= 448 * 2^e (448 is the largest e4m3 value), kept in
// [kScaleEMin, kScaleEMax].  A power of two costs no precision (the codes are
// floating point) and lets a block's scale grow later by moving exponents:
// a code loses bits only where it falls below the smallest normal code.
#pragma once

#include "common.cuh"

namespace gqa {
namespace {

constexpr int kScaleEMin = -60;
constexpr int kScaleEMax = 60;

// Two e4m3 codes (low byte first) -> two fp16 values, exact.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t two) {
  uint32_t d;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(d) : "h"((unsigned short)two));
  return d;
}
// Two fp32 values -> two e4m3 codes (lo in the low byte), round to nearest
// even; beyond +-448 saturates, NaN stays NaN.
__device__ __forceinline__ uint32_t f32x2_to_e4m3x2(float lo, float hi) {
  unsigned short d;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(hi), "f"(lo));
  return d;
}
__device__ __forceinline__ float2 f16x2_to_f32x2(uint32_t h) {
  float2 r;
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
      "cvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "r"(h));
  return r;
}

// The scale of a block whose largest finite magnitude is amax (>= 0).
__device__ __forceinline__ float block_scale(float amax) {
  const uint32_t bits = __float_as_uint(amax);
  // amax = 1.m * 2^(E-127) <= 1.75 * 2^8 * 2^e  <=>  e >= E-127-8, one more if m > .75
  int e = (int)(bits >> 23) - 127 - 8 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0);
  e = min(max(e, kScaleEMin), kScaleEMax);
  return __uint_as_float((uint32_t)(e + 127) << 23);
}

}  // namespace
}  // namespace gqa
