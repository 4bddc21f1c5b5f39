// int8.h -- INT8 rows: one fp32 scale a row, scale = amax * fp32(1 / 127) and
// code = the integer nearest to value / scale (ties to even).
#pragma once

#include "device.h"

namespace epk {

// Magnitude bits of a float: ordered like the magnitudes, infinities and NaN
// above every finite value, so one unsigned maximum also tells whether a row
// holds a value that is not finite.
__device__ __forceinline__ uint32_t magnitude_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }
constexpr uint32_t kInfBits = 0x7F800000u;

// Scale of a row (or of an FP8 block) whose largest magnitude is amax, from
// the quotient of amax and the format's largest code: 1 for a row of zeros,
// NaN for one that holds a value that is not finite (its codes are then 0, so
// what it stands for is NaN, not a plausible number).  The scale stays at
// 2^-126 or above, so that its reciprocal is finite.
__device__ __forceinline__ float scale_of(uint32_t amax_bits, float quotient) {
  if (amax_bits >= kInfBits) return __uint_as_float(0x7FC00000u);
  if (amax_bits == 0u) return 1.0f;
  return fmaxf(quotient, 1.17549435e-38f);
}
// INT8: times the rounded 1/127 -- a scale is free to be a last bit off, the
// codes are decided against it -- FP8: the division its format is defined by.
__device__ __forceinline__ float int8_scale(uint32_t amax_bits) {
  return scale_of(amax_bits, __uint_as_float(amax_bits) * (1.0f / 127.0f));
}
__device__ __forceinline__ float fp8_scale(uint32_t amax_bits) {
  return scale_of(amax_bits, __uint_as_float(amax_bits) / 448.0f);
}

// The integer nearest to the exact quotient y / s, ties to even, at most 127
// in magnitude; inv = 1 / s.  y * inv is within 2^-16 of the quotient, so its
// rounding is at most one off, and only next to a tie; r = y - q*s is exact
// there (q has 7 bits, and |r| <= s/2 up to that error), and comparing it with
// s / 2 settles it.
__device__ __forceinline__ int32_t int8_code(float y, float s, float inv) {
  float q = rintf(y * inv);
  const float r = __builtin_fmaf(-q, s, y), half = 0.5f * s, a = fabsf(r);
  const int32_t qi = (int32_t)q;
  const int32_t step = a > half || (a == half && (qi & 1)) ? (r > 0.0f ? 1 : -1) : 0;
  const int32_t c = qi + step;
  return c > 127 ? 127 : c < -127 ? -127 : c;
}

// Eight codes in memory order.
__device__ __forceinline__ u32x2 int8_codes(const float y[8], float s, float inv) {
  uint32_t w[2] = {0u, 0u};
#pragma unroll
  for (int c = 0; c < 8; ++c) w[c >> 2] |= (uint32_t)(int8_code(y[c], s, inv) & 0xFF) << (8 * (c & 3));
  return u32x2{w[0], w[1]};
}

}  // namespace epk
