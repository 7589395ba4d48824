// Codes and scales of the 8-bit K/V cache, shared by the kernels that write, read and attend to it.
//
// A cache holds e4m3 codes [num_blocks, Hkv, bs, d] beside fp32 scales [num_blocks, Hkv, bs / sb]: `sb` consecutive
// tokens of a page share one scale per KV head, and a value is code * scale.  The library's own scales are powers of two:
// a code then changes exactly when a block's scale does (but for what falls among e4m3's subnormals), e4m3 being a
// floating type such a scale costs no precision, and a value is exact in bf16.
#pragma once

#include "common.cuh"
#include "page_grid.cuh"

namespace ts {

constexpr float kCodeMax = 448.f;                                  // e4m3's largest magnitude
constexpr float kScaleLo = 9.094947017729282e-13f;                 // 2^-40
constexpr float kScaleHi = 1.099511627776e12f;                     // 2^40

// Scales as the kernels read them: a caller's own that is zero, negative, NaN or out of range is clamped.
__device__ __forceinline__ float scale_in_range(float s) { return fminf(fmaxf(s, kScaleLo), kScaleHi); }

// Exponent of a block's scale: the smallest e in [-40, 40] with amax <= 448 * 2^e (amax >= 0; infinity gives 40).
// amax lies in [2^x, 2^(x+1)), and 448 * 2^(x-8) = 1.75 * 2^x.
__device__ __forceinline__ int scale_exponent(float amax) {
  const uint32_t bits = __float_as_uint(amax);
  const int x = static_cast<int>(bits >> 23) - 127;
  const int e = (bits & 0x7FFFFFu) <= 0x600000u ? x - 8 : x - 7;  // 0x600000: the fraction of 1.75
  return max(kGridLo, min(kGridHi, e));
}

// Two codes (low byte first) <-> two values.  To nearest even, saturated to +-448, NaN stays NaN; decoding is exact.
__device__ __forceinline__ uint32_t encode_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t encode_e5m2x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t decode_e4m3x2_f16(uint32_t two) {  // -> f16x2
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(two)));
  return r;
}
__device__ __forceinline__ float2 half2_to_float2(uint32_t h) {
  float2 f;
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
      : "=f"(f.x), "=f"(f.y)
      : "r"(h));
  return f;
}
__device__ __forceinline__ float2 decode_e4m3x2(uint32_t two) { return half2_to_float2(decode_e4m3x2_f16(two)); }
__device__ __forceinline__ float decode_e4m3(uint32_t one) { return decode_e4m3x2(one & 0xFFu).x; }

}  // namespace ts
