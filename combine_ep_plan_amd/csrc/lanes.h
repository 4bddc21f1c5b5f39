// lanes.h -- sums and maxima over a wave or a workgroup of up to 16 waves
// (gfx950): four DPP moves inside each 16-lane row, then the permlane16 and
// permlane32 swaps; no LDS inside a wave.
#pragma once

#include "route_impl.h"

namespace epk {

// v of lane l ^ 1, ^ 2, then of the mirrored lane in the half row and the row:
// a reduction over these four steps leaves every lane its row's result.
template <int CTRL>
__device__ __forceinline__ double dpp_d(double v) {
  const uint64_t b = (uint64_t)__double_as_longlong(v);
  return __longlong_as_double((int64_t)join(dpp<CTRL>((uint32_t)b), dpp<CTRL>((uint32_t)(b >> 32))));
}

__device__ __forceinline__ double row_sum(double v) {
  v += dpp_d<kDppXor1>(v);
  v += dpp_d<kDppXor2>(v);
  v += dpp_d<kDppHalfMirror>(v);
  v += dpp_d<kDppMirror>(v);
  return v;
}

__device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }

__device__ __forceinline__ uint32_t row_max(uint32_t v) {
  v = umax(v, dpp<kDppXor1>(v));
  v = umax(v, dpp<kDppXor2>(v));
  v = umax(v, dpp<kDppHalfMirror>(v));
  v = umax(v, dpp<kDppMirror>(v));
  return v;
}

// Across the four rows: a swap of a register with itself leaves, in its two
// results, the values of the even and odd rows (halves), so combining the two
// needs no selection.
__device__ __forceinline__ void swap16(double v, double &a, double &b) {
  const uint64_t w = (uint64_t)__double_as_longlong(v);
  const auto lo = __builtin_amdgcn_permlane16_swap((uint32_t)w, (uint32_t)w, false, false);
  const auto hi = __builtin_amdgcn_permlane16_swap((uint32_t)(w >> 32), (uint32_t)(w >> 32), false, false);
  a = __longlong_as_double((int64_t)join(lo[0], hi[0]));
  b = __longlong_as_double((int64_t)join(lo[1], hi[1]));
}
__device__ __forceinline__ void swap32(double v, double &a, double &b) {
  const uint64_t w = (uint64_t)__double_as_longlong(v);
  const auto lo = __builtin_amdgcn_permlane32_swap((uint32_t)w, (uint32_t)w, false, false);
  const auto hi = __builtin_amdgcn_permlane32_swap((uint32_t)(w >> 32), (uint32_t)(w >> 32), false, false);
  a = __longlong_as_double((int64_t)join(lo[0], hi[0]));
  b = __longlong_as_double((int64_t)join(lo[1], hi[1]));
}

__device__ __forceinline__ double join_rows_sum(double v) {
  double a, b;
  swap16(v, a, b);
  v = a + b;
  swap32(v, a, b);
  return a + b;
}

__device__ __forceinline__ uint32_t join_rows_max(uint32_t v) {
  auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
  v = umax(r[0], r[1]);
  r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  return umax(r[0], r[1]);
}

__device__ __forceinline__ double wave_sum(double v) { return join_rows_sum(row_sum(v)); }
__device__ __forceinline__ uint32_t wave_max(uint32_t v) { return join_rows_max(row_max(v)); }

}  // namespace epk
