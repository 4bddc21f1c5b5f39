// gemm_int8.hip -- grouped GEMM of the experts on INT8 operands, gfx950 MFMA.
//
// A row of X and a row n of an expert's [N, K] weights are int8 codes with one
// fp32 scale each, so for every group of receive rows that share a weight
// matrix (see gemm.hip)
//   Y[row][n] = bf16( SX[row] * SW[n] * sum_c X[row][c] * W[n][c] ).
// The sum runs in 32-bit integers on v_mfma_i32_32x32x32_i8 and is exact:
// |codes| <= 128 and K <= 131071 keep it below 2^31.  The scales do not depend
// on c, so they are applied once, in the epilogue, in fp32, and the value is
// rounded once to bf16.
//
// SwiGLU store: weight rows interleave gate (even) and up (odd).  The loader
// puts row 2l + j of every 64 weight rows at LDS row 32j + l, so the gate and
// the up of one output are the same element of two accumulators of one lane:
// silu(gate) * up is formed from the fp32 values and rounded once (the bf16
// and FP8 kernels round gate and up to bf16 first).
//
// k_grouped_gemm_i8: 128 x 128 tiles, 256 threads, two workgroups a CU; four
// waves in 2 x 2, each 2 x 2 accumulators of 32 x 32; slabs of 128 bytes of
// K, double-buffered in LDS with the chunk swizzle of gemm_common.h.
#include "gemm_common.h"

namespace epk {

typedef int32_t i32x4 __attribute__((ext_vector_type(4)));
typedef int32_t i32x16 __attribute__((ext_vector_type(16)));

constexpr int kI8Slab = 128;  // bytes of K in a slab row

// Weight row of the tile that LDS row r holds (SwiGLU: gates, then ups, of 64).
template <bool GLU>
__device__ __forceinline__ int weight_row(int r) {
  return GLU ? (r & ~63) | ((r & 31) << 1) | ((r >> 5) & 1) : r;
}

// silu(g) * u in fp32: the hardware reciprocal and exponential (far below the
// bf16 rounding); below g = -64, where the reciprocal heads for the subnormal
// range, g * u * e^g in double (as the bf16 kernels' store).
__device__ __forceinline__ float silu_mul(float g, float u) {
  if (g < -64.0f) return (float)((double)g * (double)u * exp((double)g));
  return g * __builtin_amdgcn_rcpf(1.0f + __expf(-g)) * u;
}

__device__ __forceinline__ uint16_t bf16_bits(float v) {
  return (uint16_t)(pack_bf16x2(v, 0.0f) & 0xFFFFu);
}

template <bool GLU>
__global__ __launch_bounds__(kGemmThreads, 2) void k_grouped_gemm_i8(
    const u32x4 *__restrict__ X, const float *__restrict__ SX, const u32x4 *__restrict__ W,
    const float *__restrict__ SW, const u32x4 *__restrict__ Wslot,
    const float *__restrict__ SWslot, const int32_t *__restrict__ tiles,
    const int32_t *__restrict__ ntiles, int32_t max_tiles, int32_t K, int32_t N, int32_t E,
    int32_t n_col_tiles, uint16_t *__restrict__ Y) {
  __shared__ u32x4 sa[2][kTileM * kChunks];
  __shared__ u32x4 sb[2][kBN * kChunks];
  __shared__ float ssx[kTileM];
  int32_t tile, ctile;
  if (!balanced_tile(ntiles, max_tiles, n_col_tiles, tile, ctile)) return;
  const int32_t n0 = ctile * kBN;
  const int32_t row0 = tiles[tile * 4 + 0], rows = tiles[tile * 4 + 1], widx = tiles[tile * 4 + 2];
  const int32_t KV = K / 16;  // 16-byte vectors per row
  const bool own = widx < E;
  const int64_t wsel = own ? widx : widx - E;
  const int32_t wrows = N - n0 < kBN ? N - n0 : kBN;
  const u32x4 *Xt = X + (int64_t)row0 * KV;
  const u32x4 *Wt = (own ? W : Wslot) + (wsel * N + n0) * KV;
  const float *SWt = (own ? SW : SWslot) + wsel * N + n0;

  const int tid = threadIdx.x, lane = tid & 63;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wv / kWavesN, wn = wv % kWavesN;
  if (tid < kTileM) ssx[tid] = SX[row0 + (tid < rows ? tid : rows - 1)];

  // Loader: slot q = tid + i * 256 of a slab is row q / 8, chunk q % 8; rows
  // past the tile's end read its last row (their products are not stored).
  // K % 64 == 0: an odd half slab at the end is read as the last 128 bytes of
  // the row, of which only the upper half is used; a row of 64 bytes (K = 64)
  // is read twice into the two halves.
  constexpr int kLoads = kTileM * kChunks / kGemmThreads;
  const int c_ld = tid & (kChunks - 1), c_src = K == 64 ? c_ld & 3 : c_ld;
  const u32x4 *pa[kLoads], *pb[kLoads];
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const int r = (tid + i * kGemmThreads) / kChunks, n = weight_row<GLU>(r);
    pa[i] = Xt + (int64_t)(r < rows ? r : rows - 1) * KV + c_src;
    pb[i] = Wt + (int64_t)(n < wrows ? n : wrows - 1) * KV + c_src;
  }
  const int KT = (K + kI8Slab - 1) / kI8Slab;
  const int last = K > kI8Slab ? KV - kChunks : 0;  // first chunk of the last slab
  const bool half = K % kI8Slab != 0;               // its lower half was done already

  i32x16 acc[kFM][kFN];
#pragma unroll
  for (int i = 0; i < kFM; ++i)
#pragma unroll
    for (int j = 0; j < kFN; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0;

  u32x4 ra[kLoads], rb[kLoads];
  auto load = [&](int kt) {
    const int c = kt + 1 < KT ? kt * kChunks : last;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) ra[i] = pa[i][c];
#pragma unroll
    for (int i = 0; i < kLoads; ++i) rb[i] = pb[i][c];
  };
  auto put = [&](int buf) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) sa[buf][swz((tid + i * kGemmThreads) / kChunks, c_ld)] = ra[i];
#pragma unroll
    for (int i = 0; i < kLoads; ++i) sb[buf][swz((tid + i * kGemmThreads) / kChunks, c_ld)] = rb[i];
  };
  load(0);
  put(0);
  __syncthreads();
  for (int kt = 0; kt < KT; ++kt) {
    const int buf = kt & 1;
    if (kt + 1 < KT) load(kt + 1);
    // step kk: 32 bytes of K, the lower half-wave's lanes hold the first 16
    for (int kk = kt + 1 == KT && half ? 2 : 0; kk < 4; ++kk) {
      const int c = kk * 2 + (lane >> 5);
      i32x4 fa[kFM], fb[kFN];
#pragma unroll
      for (int i = 0; i < kFM; ++i)
        fa[i] = __builtin_bit_cast(i32x4, sa[buf][swz(wm * kWTM + i * 32 + (lane & 31), c)]);
#pragma unroll
      for (int j = 0; j < kFN; ++j)
        fb[j] = __builtin_bit_cast(i32x4, sb[buf][swz(wn * kWTN + j * 32 + (lane & 31), c)]);
#pragma unroll
      for (int i = 0; i < kFM; ++i)
#pragma unroll
        for (int j = 0; j < kFN; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fa[i], fb[j], acc[i][j], 0, 0, 0);
    }
    if (kt + 1 < KT) put(buf ^ 1);
    __syncthreads();
  }

  // accumulator r of a lane: row (r / 4) * 8 + (lane / 32) * 4 + r % 4, column lane % 32
  const int32_t NO = GLU ? N / 2 : N;
  float sw[kFN];
#pragma unroll
  for (int j = 0; j < kFN; ++j) {
    const int n = weight_row<GLU>(wn * kWTN + j * 32 + (lane & 31));
    sw[j] = SWt[n < wrows ? n : wrows - 1];
  }
#pragma unroll
  for (int i = 0; i < kFM; ++i)
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      const int rr = wm * kWTM + i * 32 + (r >> 2) * 8 + (lane >> 5) * 4 + (r & 3);
      if (rr >= rows) continue;
      const float sx = ssx[rr];
      uint16_t *y = Y + (int64_t)(row0 + rr) * NO;
      if constexpr (GLU) {
        const int col = (n0 + wn * kWTN) / 2 + (lane & 31);
        const float g = (float)acc[i][0][r] * (sx * sw[0]), u = (float)acc[i][1][r] * (sx * sw[1]);
        if (col < NO) y[col] = bf16_bits(silu_mul(g, u));
      } else {
#pragma unroll
        for (int j = 0; j < kFN; ++j) {
          const int col = n0 + wn * kWTN + j * 32 + (lane & 31);
          if (col < N) y[col] = bf16_bits((float)acc[i][j][r] * (sx * sw[j]));
        }
      }
    }
}

bool gemm_int8_fits(const Geometry &g, int32_t K, int32_t N) {
  // blocks * threads of a launch stay below 2^32
  const int64_t ncol = (N + kBN - 1) / kBN;
  return K <= kI8MaxK && gemm_grid_blocks(gemm_max_tiles(g), 1) * ncol <= UINT32_MAX / kGemmThreads;
}

hipError_t launch_grouped_gemm_int8(const Geometry &g, const Workspace &ws, const uint8_t *x,
                                    const float *sx, const uint8_t *w, const float *sw,
                                    const uint8_t *wslot, const float *swslot, int32_t K,
                                    int32_t N, uint16_t *y, bool glu, hipStream_t s) {
  const int32_t max_tiles = gemm_max_tiles(g);
  if (g.n == 0 || max_tiles == 0) return hipSuccess;
  const hipError_t e = launch_gemm_tiles(g, ws, wslot != nullptr, false, max_tiles, s);
  if (e != hipSuccess) return e;
  const int32_t ncol = (N + kBN - 1) / kBN;
  const unsigned grid = (unsigned)gemm_grid_blocks(max_tiles, ncol);
#define I8_ARGS                                                                              \
  dim3(grid), dim3(kGemmThreads), 0, s, reinterpret_cast<const u32x4 *>(x), sx,              \
      reinterpret_cast<const u32x4 *>(w), sw, reinterpret_cast<const u32x4 *>(wslot), swslot, \
      ws.gemm_tiles, ws.gemm_ntiles, max_tiles, K, N, g.E, ncol, y
  if (glu) hipLaunchKernelGGL(k_grouped_gemm_i8<true>, I8_ARGS);
  else hipLaunchKernelGGL(k_grouped_gemm_i8<false>, I8_ARGS);
#undef I8_ARGS
  return hipGetLastError();
}

}  // namespace epk
