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
// one 16-byte vector).  Maxima are taken on the bf16 bits, two at a time: of a row
// by lane moves over 16 lanes, of a column over the thread's eight rows, the
// wave's four row groups and, through LDS, the four waves.  One thread forms a
// row's or column's scale and its reciprocal for all (a division takes as long as
// two values' codes).  Codes of a row go out from registers (128 bytes a row);
// codes of a column are packed eight rows at a time into LDS, its 8-byte chunks
// permuted so that neither side meets a bank twice, and leave as 128-byte lines.
// Bound by memory (16384 x 4096 rows and columns 53 us, 5.1 TB/s); few tiles by the
// latency of one (1536 x 4096 squares, 384 tiles, 7.3 us).
#include "ep_internal.h"
#include "rows.h"

namespace epk {

constexpr int kQT = 128;            // tile
constexpr int kQThreads = 256;

typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));

// Two 16-bit maxima at once (of bf16 magnitudes, which order like their bits).
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, a),
                                                                __builtin_bit_cast(u16x2, b)));
}
__device__ __forceinline__ uint32_t join_rows_max2(uint32_t v) {
  auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
  v = max2(r[0], r[1]);
  r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  return max2(r[0], r[1]);
}
__device__ __forceinline__ uint32_t row_max2(uint32_t v) {
  v = max2(v, dpp<kDppXor1>(v));
  v = max2(v, dpp<kDppXor2>(v));
  v = max2(v, dpp<kDppHalfMirror>(v));
  return max2(v, dpp<kDppMirror>(v));
}

// A block's scale and its reciprocal; 0 for that where the codes divide (tiny and
// huge scales, and the NaN of a block that holds a value that is not finite).
__device__ __forceinline__ f32x2 scale_pair(uint32_t amax_bits, bool pow2) {
  const float s = fp8_block_scale(amax_bits, pow2);
  return f32x2{s, s >= 0x1p-80f && s <= 0x1p80f ? 1.0f / s : 0.0f};
}

// Codes of eight values of blocks with these scales: y / s correctly rounded
// (fp8_quotients).  No clamp where s is not tiny: |y| <= amax, so the quotient is
// 448 and a rounding at most, whose code is 448's.
__device__ __forceinline__ u32x2 codes8(const float y[8], f32x2 s) {
  float q[8];
  if (s.y != 0.0f) {
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      const float q0 = y[c] * s.y;
      q[c] = copysignf(__builtin_fmaf(__builtin_fmaf(-q0, s.x, y[c]), s.y, q0), y[c]);
    }
  } else {
#pragma unroll
    for (int c = 0; c < 8; ++c) q[c] = s.x == s.x ? fminf(fmaxf(y[c] / s.x, -448.0f), 448.0f) : 0.0f;
  }
  return pack_fp8(q);
}

template <bool SQUARE>
__global__ __launch_bounds__(kQThreads) void k_quantize_2d(const u32x4 *__restrict__ x, int32_t R,
                                                           int32_t C, uint8_t *__restrict__ codes,
                                                           float *__restrict__ scales,
                                                           uint8_t *__restrict__ codes_t,
                                                           float *__restrict__ scales_t, bool pow2) {
  __shared__ u32x4 s_max[4][16];                // of the waves' columns
  __shared__ f32x2 s_row[kQT], s_col[kQT];      // scales and reciprocals
  __shared__ u32x4 s_t[kQT * 8];                // [column][8-byte chunk of rows, two to a vector]
  static_assert(alignof(decltype(s_t)) >= 16, "read as 16-byte vectors");
  const int tid = threadIdx.x, cl = tid & 15, rl = tid >> 4, wv = tid >> 6;
  const int32_t nb = C / kQT, tr = blockIdx.x / nb, tc = blockIdx.x - tr * nb;
  const int64_t Rp = (int64_t)((R + kQT - 1) / kQT) * kQT;
  const int32_t row = tr * kQT + rl * 8;   // this thread's rows: row .. row + 7
  const int64_t V = C / 8, col = (int64_t)tc * 16 + cl;
  u32x4 v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
    v[i] = row + i < R ? load_stream(x + (row + i) * V + col) : u32x4{0u, 0u, 0u, 0u};
  uint32_t mr[4];                  // of rows 2 k and 2 k + 1
  u32x4 mc = {0u, 0u, 0u, 0u};     // of columns 2 k and 2 k + 1
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    uint32_t t[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const u32x4 m = v[2 * k + h] & 0x7FFF7FFFu;
#pragma unroll
      for (int w = 0; w < 4; ++w) mc[w] = max2(mc[w], m[w]);
      t[h] = max2(max2(m.x, m.y), max2(m.z, m.w));
    }
    mr[k] = max2((t[0] & 0xFFFFu) | (t[1] << 16), (t[0] >> 16) | (t[1] & 0xFFFF0000u));
  }
  f32x2 sq = {1.0f, 1.0f};   // SQUARE: the tile's
  if constexpr (SQUARE) {
    uint32_t m = join_rows_max2(row_max2(max2(max2(mr[0], mr[1]), max2(mr[2], mr[3]))));
    if ((tid & 63) == 0) s_max[wv][0].x = m;
    __syncthreads();
    m = max2(max2(s_max[0][0].x, s_max[1][0].x), max2(s_max[2][0].x, s_max[3][0].x));
    sq = scale_pair(umax(m & 0xFFFF0000u, m << 16), pow2);
    if (tid == 0) {
      if (scales) scales[(int64_t)tr * nb + tc] = sq.x;
      if (scales_t) scales_t[(int64_t)tc * (Rp / kQT) + tr] = sq.x;
    }
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      mr[k] = row_max2(mr[k]);
      mc[k] = join_rows_max2(mc[k]);   // the wave's four row groups
    }
    if ((tid & 63) < 16) s_max[wv][cl] = mc;
    if (cl < 8) {   // lane cl has the scale of row cl
      const uint32_t m = cl < 4 ? (cl < 2 ? mr[0] : mr[1]) : (cl < 6 ? mr[2] : mr[3]);
      const f32x2 s = scale_pair((cl & 1) ? m & 0xFFFF0000u : m << 16, pow2);
      s_row[rl * 8 + cl] = s;
      if (scales && row + cl < R) scales[(int64_t)(row + cl) * nb + tc] = s.x;
    }
    __syncthreads();
    if (tid < kQT && codes_t) {
      const uint32_t *const m4 = reinterpret_cast<const uint32_t *>(&s_max[0][0]) + (tid >> 1);
      const uint32_t m = max2(max2(m4[0], m4[64]), max2(m4[128], m4[192]));
      const f32x2 s = scale_pair((tid & 1) ? m & 0xFFFF0000u : m << 16, pow2);
      s_col[tid] = s;
      scales_t[((int64_t)tc * kQT + tid) * (Rp / kQT) + tr] = s.x;
    }
    __syncthreads();
  }
  u32x2 *const out = reinterpret_cast<u32x2 *>(codes);
  if (codes) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float f[8];
      unpack8(v[i], f);
      const u32x2 q = codes8(f, SQUARE ? sq : s_row[rl * 8 + i]);
      if (row + i < R) out[(row + i) * V + col] = q;
    }
  }
  if (!codes_t) return;
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    float f[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = (c & 1) ? bf16_hi(v[i][c >> 1]) : bf16_lo(v[i][c >> 1]);
    reinterpret_cast<u32x2 *>(s_t)[(cl * 8 + c) * 16 + (rl ^ cl)] =   // chunk rl, permuted by the column's group
        codes8(f, SQUARE ? sq : s_col[cl * 8 + c]);
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int k = j * kQThreads + tid, c = k >> 3, p = k & 7;   // column, 16-byte piece of its 128 rows
    const int g = (c >> 3) & 15;
    const u32x4 d = s_t[c * 8 + (p ^ (g >> 1))];
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
