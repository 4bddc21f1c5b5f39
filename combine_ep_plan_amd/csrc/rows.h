// rows.h -- what the kernels over whole rows of channels share (norm.hip,
// layernorm.hip): vectors of eight values as they are stored, reductions over
// the threads of a row, FP8 codes of values in registers, and the shape of a
// launch over rows.
#pragma once

#include "device.h"
#include "int8.h"
#include "lanes.h"

namespace epk {

enum Quant : int32_t { kQuantNone = 0, kQuantFp8 = 1, kQuantFp8Pow2 = 2, kQuantInt8 = 3 };

// Eight values of a bf16 or fp32 row as they are stored.
template <typename T>
struct Raw8 {
  u32x4 v[sizeof(T) / 2];
};

template <typename T, bool NT>
__device__ __forceinline__ Raw8<T> load_raw(const void *p, int64_t v) {
  Raw8<T> r;
  const u32x4 *q = static_cast<const u32x4 *>(p) + v * (int)(sizeof(T) / 2);
#pragma unroll
  for (int i = 0; i < (int)(sizeof(T) / 2); ++i) r.v[i] = NT ? load_stream(q + i) : q[i];
  return r;
}

template <typename T>
__device__ __forceinline__ void unpack_raw(const Raw8<T> &r, float f[8]) {
  if constexpr (sizeof(T) == 2) {
    unpack8(r.v[0], f);
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      f[4 * i] = __uint_as_float(r.v[i].x);
      f[4 * i + 1] = __uint_as_float(r.v[i].y);
      f[4 * i + 2] = __uint_as_float(r.v[i].z);
      f[4 * i + 3] = __uint_as_float(r.v[i].w);
    }
  }
}

template <typename T>
__device__ __forceinline__ void load8(const void *p, int64_t v, float f[8]) {
  unpack_raw(load_raw<T, false>(p, v), f);
}

template <typename T>
__device__ __forceinline__ void store8(void *p, int64_t v, const float f[8]) {
  if constexpr (sizeof(T) == 2) {
    static_cast<u32x4 *>(p)[v] = pack8(f);
  } else {
    static_cast<f32x4 *>(p)[2 * v] = f32x4{f[0], f[1], f[2], f[3]};
    static_cast<f32x4 *>(p)[2 * v + 1] = f32x4{f[4], f[5], f[6], f[7]};
  }
}

__device__ __forceinline__ void load_weight8(const void *w, int32_t fp32, int64_t v, float f[8]) {
  if (fp32) load8<float>(w, v, f);
  else load8<uint16_t>(w, v, f);
}

// rstd of a row from its sum of squares: the hardware's fp64 reciprocal square
// root (about 2^-26) and two Newton steps, then one rounding to fp32.
__device__ __forceinline__ float rstd_of(double ss, double inv_h, double eps) {
  const double a = __builtin_fma(ss, inv_h, eps);
  double r = __builtin_amdgcn_rsq(a);
#pragma unroll
  for (int i = 0; i < 2; ++i) r = __builtin_fma(0.5 * r, __builtin_fma(-a * r, r, 1.0), r);
  // an infinite or NaN sum: 1 / sqrt of it
  return a < 1e300 ? (float)r : (float)(1.0 / sqrt(a));
}

// Maximum of m (and sum of v) over the workgroup (up to 16 waves) or, WAVE,
// over the wave.
template <bool WAVE>
__device__ __forceinline__ void row_reduce(uint32_t &m) {
  m = wave_max(m);
  if constexpr (!WAVE) {
    __shared__ uint32_t s_max[16];
    const int lane = threadIdx.x & 63, nw = blockDim.x >> 6;
    if (lane == 0) s_max[threadIdx.x >> 6] = m;
    __syncthreads();
    m = row_max((lane & 15) < nw ? s_max[lane & 15] : 0u);
  }
}
template <bool WAVE>
__device__ __forceinline__ void row_reduce(double &v, uint32_t &m) {
  v = wave_sum(v);
  m = wave_max(m);
  if constexpr (!WAVE) {
    __shared__ double s_sum[16];
    __shared__ uint32_t s_max[16];
    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6, nw = blockDim.x >> 6;
    if (lane == 0) {
      s_sum[wv] = v;
      s_max[wv] = m;
    }
    __syncthreads();
    const int i = lane & 15;  // every 16-lane row reduces the waves' results
    v = row_sum(i < nw ? s_sum[i] : 0.0);
    m = row_max(i < nw ? s_max[i] : 0u);
  }
}

// Scale of an FP8 block from the bits of its largest magnitude: amax / 448, or
// with pow2 the power of two at or above it.
__device__ __forceinline__ float fp8_block_scale(uint32_t amax_bits, bool pow2) {
  float s = fp8_scale(amax_bits);
  if (pow2 && amax_bits != 0u && amax_bits < kInfBits) {
    const uint32_t b = __float_as_uint(s);   // subnormal ones end at 2^-126
    if (b & 0x007FFFFFu) s = __uint_as_float((b & 0x7F800000u) + 0x00800000u);
  }
  return s;
}

// The correctly rounded quotients y / s within e4m3's range, without a division
// each: with inv = 1 / s correctly rounded, q = y * inv corrected once by its
// exact remainder is y / s rounded (Markstein, "Computation of elementary
// functions on the IBM RISC System/6000 processor", 1990), where nothing
// underflows: blocks of tiny values divide.
__device__ __forceinline__ void fp8_quotients(const float y[8], float s, float q[8]) {
  if (s >= 0x1p-80f && s <= 0x1p80f) {
    const float inv = 1.0f / s;
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      const float q0 = y[c] * inv;
      // (a quotient of -0 would come back +0)
      q[c] = copysignf(__builtin_fmaf(__builtin_fmaf(-q0, s, y[c]), inv, q0), y[c]);
    }
  } else {
#pragma unroll
    for (int c = 0; c < 8; ++c) q[c] = y[c] / s;
  }
#pragma unroll
  for (int c = 0; c < 8; ++c) q[c] = fminf(fmaxf(q[c], -448.0f), 448.0f);
}

__device__ __forceinline__ u32x2 pack_fp8(const float q[8]) {
  uint32_t w0 = __builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], 0, false);
  w0 = __builtin_amdgcn_cvt_pk_fp8_f32(q[2], q[3], w0, true);
  uint32_t w1 = __builtin_amdgcn_cvt_pk_fp8_f32(q[4], q[5], 0, false);
  w1 = __builtin_amdgcn_cvt_pk_fp8_f32(q[6], q[7], w1, true);
  return u32x2{w0, w1};
}

// FP8 codes of eight values of y whose 128-channel block spans 16 lanes; the
// FP8 dispatch's recipe (quantize_fp8_vec in dispatch.hip) on fp32 values.
__device__ __forceinline__ u32x2 fp8_codes(const float y[8], float *scale, bool pow2) {
  uint32_t a = 0;
#pragma unroll
  for (int c = 0; c < 8; ++c) a = umax(a, magnitude_bits(y[c]));
  a = row_max(a);
  const float s = fp8_block_scale(a, pow2);
  *scale = s;
  if (a >= kInfBits) return u32x2{0u, 0u};
  float q[8];
  fp8_quotients(y, s, q);
  return pack_fp8(q);
}

// Workgroups of a launch over rows, RPB rows each: a launch counts its threads
// in 32 bits, so many rows spread over the grid's second dimension too.
constexpr int kRowWaves4 = 4;  // rows of a workgroup with a wave to a row
inline dim3 row_grid(int64_t rows, bool wave) {
  const int64_t blocks = wave ? (rows + kRowWaves4 - 1) / kRowWaves4 : rows;
  const int64_t gx = blocks < (1 << 20) ? blocks : 1 << 20;
  return dim3((unsigned)gx, (unsigned)((blocks + gx - 1) / gx));
}
// This thread's row, its place in it and the threads that share the row.
template <bool WAVE>
__device__ __forceinline__ int64_t my_row(int &sub, int &step) {
  const int64_t b = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
  sub = WAVE ? threadIdx.x & 63 : threadIdx.x;
  step = WAVE ? 64 : blockDim.x;
  return WAVE ? b * kRowWaves4 + (threadIdx.x >> 6) : b;
}

// Threads of a row of V vectors (V <= 4096) and vectors a thread.
struct RowShape {
  bool wave;
  int threads, vpt;
};
RowShape row_shape(int64_t rows, int32_t V);  // norm.hip
// F(VPT, WAVE) for a shape
#define EP_ROW_SWITCH(sh, F)                    \
  do {                                          \
    if (sh.wave && sh.vpt == 1) F(1, true);     \
    else if (sh.wave && sh.vpt == 2) F(2, true); \
    else if (sh.wave) F(4, true);               \
    else if (sh.vpt == 1) F(1, false);          \
    else if (sh.vpt == 2) F(2, false);          \
    else F(4, false);                           \
  } while (0)

// Threads of a row of a norm's backward, vectors a thread, rows a workgroup takes
// at a time (narrow rows share one, so that there are few partial rows of the
// weight's gradient).
struct BwdShape {
  int threads, vpt, rows;
};
inline BwdShape bwd_shape(int32_t V) {
  BwdShape b;
  b.threads = V <= 1024 ? (V + 63) / 64 * 64 : 1024;
  b.vpt = V <= b.threads ? 1 : V <= 2 * b.threads ? 2 : 4;
  b.rows = b.threads <= 256 ? 512 / b.threads : 1;
  return b;
}

}  // namespace epk
