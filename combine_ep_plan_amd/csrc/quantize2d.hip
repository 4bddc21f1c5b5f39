// quantize2d.hip -- a bf16 matrix to e4m3 codes and those of its transpose, on
// gfx950: what the FP8 products with a scale per block of 128 read (linear_fp8.hip).
//
// For a [R, C] matrix, with scale = amax / 448 over a block and code = e4m3 of
// value / scale:
//   ROWS     codes with a scale per row and 128 channels; transposed codes
//            [C, Rp] with a scale per channel and 128 rows (the operands of a
//            training step's data and weight gradients)
//   SQUARE   one scale per 128 x 128 square, for codes and transposed codes alike
//            (weights: the product and the data gradient read the same values)
// Rp is R rounded up to 128; the transposed codes past R are zeros.
//
// A workgroup takes a 128 x 128 tile, so that every block is its own: the tile
// is read once into registers, a thread holding an 8 x 8 square (eight rows of
// one 16-byte vector).  Row maxima are lane moves over 16 lanes; column maxima
// combine a thread's eight rows, lane moves over the wave's four row groups, then
// the four waves through LDS.  Codes of a row go out from registers (128 bytes a
// row); codes of a column are packed eight rows at a time into LDS, its 8-byte
// chunks permuted so that neither side meets a bank twice, and leave as 128-byte
// lines.  Bound by memory: 2 bytes read, 1 written a form.
#include "ep_internal.h"
#include "rows.h"

namespace epk {

constexpr int kQT = 128;            // tile
constexpr int kQThreads = 256;

__device__ __forceinline__ uint32_t max_bits8(const float f[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int c = 0; c < 8; ++c) m = umax(m, magnitude_bits(f[c]));
  return m;
}

// Quotients of values whose block holds one that is not finite: zeros (its
// scale is NaN).
__device__ __forceinline__ void quotients_or_zero(const float y[8], float s, float q[8]) {
  fp8_quotients(y, s, q);
  if (s != s) {
#pragma unroll
    for (int c = 0; c < 8; ++c) q[c] = 0.0f;
  }
}

template <bool SQUARE>
__global__ __launch_bounds__(kQThreads) void k_quantize_2d(const u32x4 *__restrict__ x, int32_t R,
                                                           int32_t C, uint8_t *__restrict__ codes,
                                                           float *__restrict__ scales,
                                                           uint8_t *__restrict__ codes_t,
                                                           float *__restrict__ scales_t, bool pow2) {
  __shared__ uint32_t s_max[4][kQT];
  __shared__ float s_scale[kQT];
  __shared__ u32x2 s_t[kQT * 16];   // [column][8-byte chunk of rows]
  const int tid = threadIdx.x, cl = tid & 15, rl = tid >> 4, wv = tid >> 6;
  const int32_t nb = C / kQT, tr = blockIdx.x / nb, tc = blockIdx.x - tr * nb;
  const int64_t Rp = (int64_t)((R + kQT - 1) / kQT) * kQT;
  const int32_t row = tr * kQT + rl * 8;   // this thread's rows: row .. row + 7
  const int64_t V = C / 8, col = (int64_t)tc * 16 + cl;
  u32x4 v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
    v[i] = row + i < R ? load_stream(x + (row + i) * V + col) : u32x4{0u, 0u, 0u, 0u};
  // maxima: of each row's vector, and of each column over the thread's rows
  uint32_t mr[8], mc[8] = {};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float f[8];
    unpack8(v[i], f);
    mr[i] = max_bits8(f);
    if constexpr (!SQUARE) {
#pragma unroll
      for (int c = 0; c < 8; ++c) mc[c] = umax(mc[c], magnitude_bits(f[c]));
    }
  }
  float sq = 1.0f;   // SQUARE: the tile's scale
  if constexpr (SQUARE) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = umax(m, mr[i]);
    m = wave_max(m);
    if ((tid & 63) == 0) s_max[wv][0] = m;
    __syncthreads();
    m = umax(umax(s_max[0][0], s_max[1][0]), umax(s_max[2][0], s_max[3][0]));
    sq = fp8_block_scale(m, pow2);
    if (tid == 0) {
      if (scales) scales[(int64_t)tr * nb + tc] = sq;
      if (scales_t) scales_t[(int64_t)tc * (Rp / kQT) + tr] = sq;
    }
  } else if (codes_t) {
#pragma unroll
    for (int c = 0; c < 8; ++c) mc[c] = join_rows_max(mc[c]);   // the wave's four row groups
    if ((tid & 63) < 16) {
#pragma unroll
      for (int c = 0; c < 8; ++c) s_max[wv][cl * 8 + c] = mc[c];
    }
    __syncthreads();
    if (tid < kQT) {
      const uint32_t m = umax(umax(s_max[0][tid], s_max[1][tid]), umax(s_max[2][tid], s_max[3][tid]));
      const float s = fp8_block_scale(m, pow2);
      s_scale[tid] = s;
      scales_t[((int64_t)tc * kQT + tid) * (Rp / kQT) + tr] = s;
    }
    __syncthreads();
  }
  u32x2 *const out = reinterpret_cast<u32x2 *>(codes);
  if (codes) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float f[8], q[8];
      unpack8(v[i], f);
      const float s = SQUARE ? sq : fp8_block_scale(row_max(mr[i]), pow2);
      quotients_or_zero(f, s, q);
      if (row + i < R) {
        out[(row + i) * V + col] = pack_fp8(q);
        if (!SQUARE && cl == 0) scales[(int64_t)(row + i) * nb + tc] = s;
      }
    }
  }
  if (!codes_t) return;
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    float f[8], q[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = (c & 1) ? bf16_hi(v[i][c >> 1]) : bf16_lo(v[i][c >> 1]);
    quotients_or_zero(f, SQUARE ? sq : s_scale[cl * 8 + c], q);
    s_t[(cl * 8 + c) * 16 + (rl ^ cl)] = pack_fp8(q);   // chunk rl, permuted by the column's group
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int k = j * kQThreads + tid, c = k >> 3, p = k & 7;   // column, 16-byte piece of its 128 rows
    const int g = (c >> 3) & 15;
    const u32x4 d = *reinterpret_cast<const u32x4 *>(&s_t[c * 16 + ((2 * p) ^ (g & ~1))]);
    *reinterpret_cast<u32x4 *>(codes_t + ((int64_t)tc * kQT + c) * Rp + (int64_t)tr * kQT + 16 * p) =
        (g & 1) ? u32x4{d.z, d.w, d.x, d.y} : d;
  }
}

hipError_t launch_quantize_2d(const Quantize2d &n, hipStream_t s) {
  if (n.R == 0) return hipSuccess;
  const unsigned tiles = (unsigned)(((n.R + kQT - 1) / kQT) * (n.C / kQT));
#define L(SQ)                                                                                         \
  hipLaunchKernelGGL((k_quantize_2d<SQ>), dim3(tiles), dim3(kQThreads), 0, s,                          \
                     reinterpret_cast<const u32x4 *>(n.x), n.R, n.C, n.codes, n.scales, n.codes_t,    \
                     n.scales_t, n.pow2)
  if (n.square) L(true);
  else L(false);
#undef L
  return hipGetLastError();
}

}  // namespace epk
