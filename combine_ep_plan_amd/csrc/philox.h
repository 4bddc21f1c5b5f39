// philox.h -- the counter-based generator of dropout: Philox4x32-10 (Salmon,
// Moraes, Dror, Shaw, "Parallel random numbers: as easy as 1, 2, 3", 2011).
// The mask is never stored: value i of a tensor stays if its 16 bits -- half
// i % 8 of the generator's four words at counter (i / 8, offset) under the key
// `seed` -- are below a threshold, so whoever knows i, seed and offset forms it
// again.  16 bits a value, not 32: ten rounds then serve eight values, and the
// probability is off by at most 2^-17, which the factor of the kept values
// takes into account.
//
// A round is two products 32 x 32 -> 64 bits (v_mad_u64_u32, a quarter of the
// vector rate): about 1.1 cycles of a SIMD a value, 30 us for 16384 x 4096
// values on 1024 SIMDs, which runs under the memory's 60 us and more.
#pragma once

#include "device.h"

namespace epk {

struct PhiloxKey {
  uint32_t k0, k1, o0, o1;
};

__device__ __forceinline__ PhiloxKey philox_key(const int32_t *rng) {
  return {(uint32_t)rng[0], (uint32_t)rng[1], (uint32_t)rng[2], (uint32_t)rng[3]};
}

__device__ __forceinline__ u32x4 philox(uint64_t block, const PhiloxKey &key) {
  uint32_t c0 = (uint32_t)block, c1 = (uint32_t)(block >> 32), c2 = key.o0, c3 = key.o1;
  uint32_t k0 = key.k0, k1 = key.k1;
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t a = (uint64_t)0xD2511F53u * c0, b = (uint64_t)0xCD9E8D57u * c2;
    c0 = (uint32_t)(b >> 32) ^ c1 ^ k0;
    c1 = (uint32_t)b;
    c2 = (uint32_t)(a >> 32) ^ c3 ^ k1;
    c3 = (uint32_t)a;
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return u32x4{c0, c1, c2, c3};
}

// Whether value c (0..7) of a block stays.
__device__ __forceinline__ bool stays(const u32x4 &bits, int c, uint32_t threshold) {
  const uint32_t w = bits[c >> 1];
  return ((c & 1) ? w >> 16 : w & 0xFFFFu) < threshold;
}

}  // namespace epk
