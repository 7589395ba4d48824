// The power-of-two grids of the page bounds and of the queries they are scored against.
//
// A vector is put on the grid 2^e with e the smallest exponent in [-40, 40] whose 255 * 2^e
// covers its largest magnitude (magnitudes are clamped to 255 * 2^40 first).  Its values are then
// whole multiples of 2^e of at most 255: eight significant bits, which bf16 holds exactly.  A
// product of a query value and a bound is a multiple of 2^(eq + eb) of at most 255^2, and a sum of
// up to 256 of them stays below 2^24 such units (255 * 255 * 256 = 16646400 < 16777216), so
// fp32 (the tensor cores' accumulators among it) holds every score exactly in any order.
#pragma once

#include <cstdint>

namespace ts {

constexpr int kGridLo = -40, kGridHi = 40;
constexpr float kGridMax = 255.f * 1099511627776.f;  // 255 * 2^40

// A finite, clamped value: NaN -> 0.
__device__ __forceinline__ float grid_clamp(float x) {
  return x != x ? 0.f : fminf(fmaxf(x, -kGridMax), kGridMax);
}

// Grid exponent of a vector whose largest magnitude is amax (finite, >= 0): amax lies in
// [2^x, 2^(x+1)), and 255 * 2^(x-7) = 1.9921875 * 2^x.
__device__ __forceinline__ int grid_exponent(float amax) {
  const uint32_t bits = __float_as_uint(amax);
  const int x = static_cast<int>(bits >> 23) - 127;
  const int e = (bits & 0x7FFFFFu) <= 0x7F0000u ? x - 7 : x - 6;  // 0x7F0000: the fraction of 1.9921875
  return max(kGridLo, min(kGridHi, e));
}

// 2^e for -126 <= e <= 127.
__device__ __forceinline__ float pow2(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }

}  // namespace ts
