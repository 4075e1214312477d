// The two E4M3 conversions of the quantizers (activations, and keys and values).
#pragma once
#include "common.hpp"

namespace nvfp4 {

// E4M3 byte of u >= 0 (or +inf): round to nearest even on the E4M3 grid,
// saturating at 448 (0x7E).
__device__ __forceinline__ uint32_t e4m3_rne_sat(float u) {
  if (!(u < 448.0f)) return 0x7Eu;                 // >= 448 or +inf
  if (u < 0.015625f) {                             // below 2^-6: grid step 2^-9
    return (uint32_t)__builtin_rintf(u * 512.0f);  // 0..8, and 8 encodes 2^-6
  }
  uint32_t b = __float_as_uint(u);
  b = (b + 0x7FFFFu + ((b >> 20) & 1u)) & 0xFFF00000u;   // keep 3 mantissa bits, RNE
  const uint32_t e = (b >> 23) - 127u + 7u;               // biased E4M3 exponent (1..15)
  return (e << 3) | ((b >> 20) & 7u);
}

// Value of a finite, non-negative E4M3 byte.
__device__ __forceinline__ float e4m3_value(uint32_t s) {
  const uint32_t e = s >> 3, m = s & 7u;
  if (e == 0) return (float)m * 0.001953125f;                      // m * 2^-9, exact
  return __uint_as_float(((e + 120u) << 23) | (m << 20));          // 2^(e-7) * (1 + m/8)
}

}  // namespace nvfp4
