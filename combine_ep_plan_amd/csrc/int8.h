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
// what it stands for is NaN, not a plausible number), and never below `least`.
__device__ __forceinline__ float scale_of(uint32_t amax_bits, float quotient, float least) {
  if (amax_bits >= kInfBits) return __uint_as_float(0x7FC00000u);
  if (amax_bits == 0u) return 1.0f;
  return fmaxf(quotient, least);
}
// INT8: times the rounded 1/127 -- a scale is free to be a last bit off, the
// codes are decided against it -- and at least 2^-126, so that its reciprocal is
// finite.  FP8: the division its format is defined by, subnormal ones too (the
// codes divide); at least the smallest float, where the quotient rounds to 0.
__device__ __forceinline__ float int8_scale(uint32_t amax_bits) {
  return scale_of(amax_bits, __uint_as_float(amax_bits) * (1.0f / 127.0f), 1.17549435e-38f);
}
__device__ __forceinline__ float fp8_scale(uint32_t amax_bits) {
  return scale_of(amax_bits, __uint_as_float(amax_bits) / 448.0f, __uint_as_float(1u));
}

// Eight codes in memory order: the integer nearest to the exact quotient y / s,
// ties to even; inv = 1 / s.  Adding 1.5 * 2^23 to y * inv in one fma leaves the
// rounded quotient in the low mantissa bits (its low byte is the code); it is
// off by one at most, and only next to a tie, since y * inv is within 2^-16 of
// the quotient.  r = y - q*s is exact (q has 7 bits and |r| stays near s/2), and
// so is 2r (s/2 is not, below 2^-125), so one comparison of twice the largest
// |r| of the eight with s tells whether any needs the settling below: a few in
// ten thousand do.  |y| <= amax keeps q within 127.
__device__ __forceinline__ u32x2 int8_codes(const float y[8], float s, float inv) {
  constexpr float kMagic = 12582912.0f;  // 1.5 * 2^23
  float t[8], worst = 0.0f;
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    t[c] = __builtin_fmaf(y[c], inv, kMagic);
    const float q = t[c] - kMagic;
    worst = fmaxf(worst, fabsf(__builtin_fmaf(-q, s, y[c])));
  }
  if (worst + worst >= s) {
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      const float q = t[c] - kMagic, r = __builtin_fmaf(-q, s, y[c]), a2 = fabsf(r + r);
      const bool odd = (__float_as_uint(t[c]) & 1u) != 0u;
      if (a2 > s || (a2 == s && odd)) t[c] += r > 0.0f ? 1.0f : -1.0f;
    }
  }
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    // v_perm_b32: bytes 0 of two words, then the two halves
    const uint32_t lo = __builtin_amdgcn_perm(__float_as_uint(t[4 * i + 1]), __float_as_uint(t[4 * i]), 0x0c0c0400u);
    const uint32_t hi = __builtin_amdgcn_perm(__float_as_uint(t[4 * i + 3]), __float_as_uint(t[4 * i + 2]), 0x04000c0cu);
    w[i] = lo | hi;
  }
  return u32x2{w[0], w[1]};
}

}  // namespace epk
