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
// Three kernels, chosen by rows an expert: k_grouped_gemm_i8_stream,
// k_grouped_gemm_i8 and k_grouped_gemm_i8_256.
//
// k_grouped_gemm_i8: 128 x 128 tiles, 256 threads, two workgroups a CU; four
// waves in 2 x 2, each 2 x 2 accumulators of 32 x 32; slabs of 128 bytes of
// K, double-buffered in LDS with the chunk swizzle of gemm_common.h.
#include <type_traits>

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

// ---------------------------------------------------------------------------
// Few rows an expert (decode): the time is streaming the weights, so nothing
// may stand in the way of loads.  A wave by itself streams 64 weight rows (two
// 32-column blocks; gates and ups for SwiGLU) and the tile's rows through a
// ring of slabs in its own part of LDS: no barriers, only waits for its own
// loads, D slabs in flight.  The loads go straight to LDS, eight lanes to a
// 128-byte row: loaded into registers in the order the MFMAs want (32 rows, 16
// bytes a lane) the same bytes take four times the address slots and the
// kernel stops at 6.1 TB/s of weights.  The weights are loaded non-temporally:
// plain loads of them stop at 6.2 TB/s on this card, non-temporal ones at 7.1.
// Decode (1024 rows, 256 experts, K = 7168, N = 2048): 560 us, 6.6 TB/s.
// SPLIT: the four waves of a workgroup share 64 columns and take a quarter of K
// each, so that a batch of few experts still fills the GPU; their integer
// partial sums are joined through LDS, exactly.

constexpr int kStreamCols = 64;
constexpr int32_t kShortRows = 64;  // row tiles of at most this only stream their weights

struct StreamTile {
  __amdgpu_buffer_rsrc_t rX, rW;
  const float *SX, *SW;  // scales of the tile's rows and columns
  uint16_t *Y;           // the tile's first row and column of outputs
  int32_t rows, wrows, K, NO, cols;  // cols: outputs of the tile
};

// A buffer resource of wave-uniform bounds, kept in scalar registers (the
// loads to LDS take no other; through a branch the compiler may lose sight of
// its uniformity).
__device__ __forceinline__ __amdgpu_buffer_rsrc_t uniform_rsrc(const void *p, int32_t bytes) {
  const uint64_t a = (uint64_t)(uintptr_t)p;
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)a);
  const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)(a >> 32));
  return __builtin_amdgcn_make_buffer_rsrc((void *)(uintptr_t)(((uint64_t)hi << 32) | lo), (short)0,
                                           __builtin_amdgcn_readfirstlane(bytes), kBufDword3);
}

// The stream's view of columns [n0, n0 + 64) of a row tile.
template <bool GLU>
__device__ __forceinline__ StreamTile stream_tile(const u32x4 *X, const float *SX, const u32x4 *Wm,
                                                  const float *SWm, uint16_t *Y, int32_t row0,
                                                  int32_t rows, int32_t n0, int32_t N, int32_t K) {
  const int32_t KV = K / 16, NO = GLU ? N / 2 : N;
  StreamTile t;
  t.rows = rows;
  t.wrows = N - n0 < kStreamCols ? N - n0 : kStreamCols;
  t.K = K;
  t.NO = NO;
  t.cols = GLU ? t.wrows / 2 : t.wrows;
  // every offset is in range by construction (rows past the end read the last
  // row); the rows span less than 2^31 bytes
  t.rX = uniform_rsrc(X + (int64_t)row0 * KV, rows * K);
  t.rW = uniform_rsrc(Wm + (int64_t)n0 * KV, t.wrows * K);
  t.SX = SX + row0;
  t.SW = SWm + n0;
  t.Y = Y + (int64_t)row0 * NO + (GLU ? n0 / 2 : n0);
  return t;
}

// 16-byte slots of a wave's ring: D slabs of 64 weight rows and 8 NX token rows.
constexpr int stream_slots(int NX, int D) { return D * (kStreamCols + 8 * NX) * kChunks; }

// Rows [m0, m0 + 8 NX) of the tile, NX 1, 2, 4 or 8; ring: the wave's
// stream_slots(NX, D).
template <bool GLU, int NX, int D, bool SPLIT>
__device__ __forceinline__ void stream_rows(const StreamTile &t, int32_t m0, int wv, int lane,
                                            u32x4 *ring, int32_t *part) {
  constexpr int LB = NX == 8 ? 2 : 1;       // 32-row blocks
  constexpr int SLAB = (kStreamCols + 8 * NX) * kChunks;
  constexpr int NL = kStreamCols / 8 + NX;  // loads of a slab
  static_assert((D - 1) * NL <= 63, "the wait counts them in six bits");
  const int h = lane >> 5, l = lane & 31;
  const int32_t K = t.K;
  const int KT = (K + kI8Slab - 1) / kI8Slab;
  const int lo = SPLIT ? KT * wv / 4 : 0, hi = SPLIT ? KT * (wv + 1) / 4 : KT;  // this wave's slabs
  const int last = K > kI8Slab ? K - kI8Slab : 0;
  const bool half = K % kI8Slab != 0;  // the last slab: only its upper half is new
  // load i fills the slots i*64 + lane: LDS row r = i*8 + lane/8, holding chunk
  // (lane % 8) ^ ((r / 2) % 8)
  uint32_t ow[kStreamCols / 8], ox[NX];
#pragma unroll
  for (int i = 0; i < kStreamCols / 8; ++i) {
    const int r = i * 8 + (lane >> 3), c = (lane & 7) ^ ((r >> 1) & 7), n = weight_row<GLU>(r);
    ow[i] = (uint32_t)((n < t.wrows ? n : t.wrows - 1) * K + (K == 64 ? c & 3 : c) * 16);
  }
#pragma unroll
  for (int i = 0; i < NX; ++i) {
    const int r = i * 8 + (lane >> 3), c = (lane & 7) ^ ((r >> 1) & 7), m = m0 + r;
    ox[i] = (uint32_t)((m < t.rows ? m : t.rows - 1) * K + (K == 64 ? c & 3 : c) * 16);
  }
#define LDS_ADDR(p) ((uint32_t)(size_t)LDS_PTR(p))
  const auto issue = [&](int kt, int buf) {
    const int so = kt + 1 < KT ? kt * kI8Slab : last;
#pragma unroll
    for (int i = 0; i < kStreamCols / 8; ++i)
      lds_load16_stream(t.rW, LDS_ADDR(&ring[buf * SLAB + i * 64]), ow[i], so);
#pragma unroll
    for (int i = 0; i < NX; ++i)
      lds_load16(t.rX, LDS_ADDR(&ring[buf * SLAB + (kStreamCols + 8 * i) * kChunks]), ox[i], so);
  };
#undef LDS_ADDR
  i32x16 acc[LB][2];
#pragma unroll
  for (int i = 0; i < LB; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0;
#pragma unroll
  for (int d = 0; d < D; ++d)
    if (lo + d < hi) issue(lo + d, d);
  int buf = 0;
  for (int kt = lo; kt < hi; ++kt) {
    // slab kt landed (the D - 1 after it may still be on their way)
    if (kt + D <= hi) asm volatile("s_waitcnt vmcnt(%0)" ::"n"((D - 1) * NL) : "memory");
    else asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    i32x4 fa[LB][4], fb[2][4];
    const u32x4 *sw_ = ring + buf * SLAB, *sx_ = sw_ + kStreamCols * kChunks;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
#pragma unroll
      for (int j = 0; j < 2; ++j) fb[j][c] = __builtin_bit_cast(i32x4, sw_[swz(j * 32 + l, 2 * c + h)]);
      // token rows that were not loaded (8 NX < 32) are rows nobody stores: any row serves
#pragma unroll
      for (int i = 0; i < LB; ++i)
        fa[i][c] = __builtin_bit_cast(i32x4, sx_[swz((i * 32 + l) & (8 * NX - 1), 2 * c + h)]);
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // read: the buffer is free
    if (kt + D < hi) issue(kt + D, buf);
    const bool tail = half && kt + 1 == KT;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      if (c < 2 && tail) continue;
#pragma unroll
      for (int i = 0; i < LB; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fa[i][c], fb[j][c], acc[i][j], 0, 0, 0);
    }
    buf = buf + 1 == D ? 0 : buf + 1;
  }

  float sw[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int n = GLU ? 2 * l + j : j * 32 + l;
    sw[j] = t.SW[n < t.wrows ? n : t.wrows - 1];
  }
  const auto store = [&](int32_t rr, int32_t v0, int32_t v1) {
    if (rr >= t.rows) return;
    const float sx = t.SX[rr];
    uint16_t *y = t.Y + (int64_t)rr * t.NO;
    const float f0 = (float)v0 * (sx * sw[0]), f1 = (float)v1 * (sx * sw[1]);
    if constexpr (GLU) {
      if (l < t.cols) y[l] = bf16_bits(silu_mul(f0, f1));
    } else {
      if (l < t.cols) y[l] = bf16_bits(f0);
      if (32 + l < t.cols) y[32 + l] = bf16_bits(f1);
    }
  };
  // accumulator r of a lane: row (r / 4) * 8 + (lane / 32) * 4 + r % 4
#pragma unroll
  for (int i = 0; i < LB; ++i) {
    if constexpr (!SPLIT) {
#pragma unroll
      for (int r = 0; r < 16; ++r)
        store(m0 + i * 32 + (r >> 2) * 8 + h * 4 + (r & 3), acc[i][0][r], acc[i][1][r]);
    } else {
#define PART(w_, j_, r_) part[(((w_) * 2 + (j_)) * 16 + (r_)) * 64 + lane]
      __syncthreads();   // the rings, and the parts of the rows before, are read
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r) PART(wv, j, r) = acc[i][j][r];
      __syncthreads();
      // wave wv finishes accumulator elements 4 wv .. 4 wv + 3
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        int32_t v[2];
#pragma unroll
        for (int j = 0; j < 2; ++j)
          v[j] = PART(0, j, wv * 4 + q) + PART(1, j, wv * 4 + q) + PART(2, j, wv * 4 + q) +
                 PART(3, j, wv * 4 + q);
        store(m0 + i * 32 + wv * 8 + h * 4 + q, v[0], v[1]);
      }
#undef PART
    }
  }
  if constexpr (SPLIT) __syncthreads();   // before the next rows' loads land in the rings
}

// Slabs in the ring by its token rows (8, 16, 32, 64).  A wave by itself idles
// when its slab is late and while it starts and ends, so more waves a compute
// unit beat deeper rings: kRingFew, 20 KB, eight waves (1024 rows on 256
// experts, K = 7168, N = 2048: 563 us against 602 with 36 KB rings of four
// slabs); kRingMore, 24 KB, six waves, where groups have some 16 rows or more.
// kRingWide: a wave's quarter of the 256 x 256 kernel's LDS.
struct RingDepth {
  int d1, d2, d4, d8;
};
constexpr RingDepth kRingFew = {2, 2, 1, 1}, kRingMore = {2, 2, 2, 1}, kRingWide = {4, 4, 3, 2};
constexpr int max_i(int a, int b) { return a > b ? a : b; }
constexpr int ring_slots(RingDepth d) {
  return max_i(max_i(stream_slots(1, d.d1), stream_slots(2, d.d2)),
               max_i(stream_slots(4, d.d4), stream_slots(8, d.d8)));
}
template <bool FEW, bool WIDE>
constexpr RingDepth ring_depth() {
  return WIDE ? kRingWide : FEW ? kRingFew : kRingMore;
}

// All rows of a tile, in passes of 64 over its weights (one, unless a busier
// expert stands among few rows); the smallest ring row count that holds them.
template <bool GLU, bool FEW, bool WIDE, bool SPLIT>
__device__ __forceinline__ void stream_all(const StreamTile &t, int wv, int lane, u32x4 *ring,
                                           int32_t *part) {
  constexpr RingDepth d = ring_depth<FEW, WIDE>();
  int32_t m0 = 0;
  for (; m0 + 32 < t.rows; m0 += 64) stream_rows<GLU, 8, d.d8, SPLIT>(t, m0, wv, lane, ring, part);
  const int32_t left = t.rows - m0;
  if (left > 16) stream_rows<GLU, 4, d.d4, SPLIT>(t, m0, wv, lane, ring, part);
  else if (left > 8) stream_rows<GLU, 2, d.d2, SPLIT>(t, m0, wv, lane, ring, part);
  else if (left > 0) stream_rows<GLU, 1, d.d1, SPLIT>(t, m0, wv, lane, ring, part);
}

// TABLE: 128-row tiles of the tile table; otherwise workgroup b takes a whole
// group (b / column tiles) of the plan, with no table to wait for -- for batches
// whose groups are small for certain.
template <bool GLU, bool FEW, bool SPLIT, bool TABLE>
__global__ __launch_bounds__(SPLIT ? 256 : 64) void k_grouped_gemm_i8_stream(
    const u32x4 *__restrict__ X, const float *__restrict__ SX, const u32x4 *__restrict__ W,
    const float *__restrict__ SW, const u32x4 *__restrict__ Wslot,
    const float *__restrict__ SWslot, TileArgs a, int32_t max_tiles, int32_t K, int32_t N,
    int32_t E, int32_t n_col_tiles, uint16_t *__restrict__ Y) {
  constexpr int kSlots = ring_slots(ring_depth<FEW, false>());
  __shared__ u32x4 ring[(SPLIT ? 4 : 1) * kSlots];
  static_assert(4 * 2 * 16 * 64 * 4 <= 4 * kSlots * 16, "the partial sums fit the rings");
  int32_t ctile, row0, rows, widx;
  if constexpr (TABLE) {
    int32_t tile;
    if (!balanced_tile(a.ws.gemm_ntiles, max_tiles, n_col_tiles, tile, ctile)) return;
    const int32_t *t = a.ws.gemm_tiles + (int64_t)tile * 4;
    row0 = t[0];
    rows = t[1];
    widx = t[2];
  } else {
    const int32_t q = blockIdx.x / n_col_tiles;
    ctile = blockIdx.x % n_col_tiles;
    if (a.g.layout == kStatic && q >= a.g.E + *a.ws.n_segments) return;
    group_of(a, q, row0, rows, widx);
    if (rows <= 0) return;
  }
  const bool own = widx < E;
  const int64_t wsel = own ? widx : widx - E;
  const StreamTile t = stream_tile<GLU>(X, SX, (own ? W : Wslot) + wsel * N * (K / 16),
                                        (own ? SW : SWslot) + wsel * N, Y, row0, rows,
                                        ctile * kStreamCols, N, K);
  const int lane = threadIdx.x & 63;
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  stream_all<GLU, FEW, false, SPLIT>(t, wv, lane, ring + wv * kSlots, reinterpret_cast<int32_t *>(ring));
}

// ---------------------------------------------------------------------------
// 256 x 256 tiles (large groups): four waves in 2 x 2, each 4 x 4 accumulators
// of 32 x 32 in the 256 accumulation registers; 128-byte slabs straight from
// global memory into LDS, rows of X in two buffers and of W in three (all 160
// KB).  A slab's two halves are multiplied one after the other; the one barrier
// a slab stands between them, where the slab's last fragments are in
// registers.  It publishes the next slab and frees this one's buffers, whose
// loads (X two slabs ahead, W, which misses the L2 more often, three) then go
// out under the second half's MFMAs.  Row tiles of at most kShortRows rows are
// streamed instead (above).

// A lane's fragments of half a slab: chunks 2s + lane / 32 of its row, s = 0, 1
// (within the half).
struct Frag2 {
  i32x4 s0, s1;
};

// Work of workgroup blockIdx.x.  Its XCD's work comes in chunks of 16
// workgroups: a block of 4 full row tiles by 4 column tiles, which run at about
// the same time on the XCD's compute units and share their row and weight slabs
// in its L2, or 16 column tiles of short row tiles, which stream weights; the two
// kinds merged in proportion, XCD x taking the blocks and the short tiles x, x +
// 8, ...  Against every XCD walking one row tile's column tiles at a time:
// 1010 -> 972 us on even groups (4096 tokens, 16 experts, top-8, K = 7168, N =
// 4096), 1711 -> 1663 us on the skewed prefill batch; other block shapes and
// chunk sizes (1 x 16 to 4 x 8, 8 to 64) fell between.
constexpr int kBlock = 4, kChunk = kBlock * kBlock;
__device__ __forceinline__ bool blocked_tile(const int32_t *__restrict__ ntiles, int32_t max_tiles,
                                             int32_t n_col_tiles, int32_t &tile, int32_t &col) {
  const int32_t nf = ntiles[1], ns = ntiles[0] - nf;
  const int32_t x = blockIdx.x % kXcds, slot = blockIdx.x / kXcds;
  const int32_t cg = (n_col_tiles + kBlock - 1) / kBlock;
  const int32_t nb = (nf + kBlock - 1) / kBlock * cg;
  const int32_t fx = x < nb ? (nb - x + kXcds - 1) / kXcds : 0;   // this XCD's blocks ...
  const int32_t sx = x < ns ? (ns - x + kXcds - 1) / kXcds : 0;   // ... and short tiles
  const int32_t n = fx + (sx * n_col_tiles + kChunk - 1) / kChunk;
  const int32_t p = slot / kChunk, i = slot % kChunk;
  if (p >= n) return false;
  const int32_t f = (int32_t)((int64_t)p * fx / n);
  if ((int32_t)((int64_t)(p + 1) * fx / n) > f) {
    const int32_t b = x + kXcds * f;
    tile = b / cg * kBlock + i % kBlock;
    col = b % cg * kBlock + i / kBlock;
    return tile < nf && col < n_col_tiles;
  }
  const int32_t q = (p - f) * kChunk + i, t = q / n_col_tiles;
  tile = max_tiles - 1 - (x + kXcds * t);
  col = q - t * n_col_tiles;
  return t < sx;
}
// Workgroups that cover it for any split of max_tiles row tiles into kinds: per
// XCD an eighth of the blocks, rounded up, and of the short tiles' chunks.
static int64_t blocked_grid(int32_t max_tiles, int64_t ncol) {
  const int64_t blocks = ((int64_t)max_tiles / kBlock + 1) * ((ncol + kBlock - 1) / kBlock);
  const int64_t chunks = (((int64_t)max_tiles / kXcds + 1) * ncol + kChunk - 1) / kChunk;
  return kXcds * kChunk * (blocks / kXcds + 1 + chunks);
}

template <int I, int NB>
__device__ __forceinline__ void mfma_i8_rows(i32x16 (&acc)[kFM2][kFN2], const Frag2 (&fa)[kFM2],
                                             const Frag2 (&fb)[kFN2]) {
  if constexpr (I < NB) {
#pragma unroll
    for (int j = 0; j < kFN2; ++j)
      acc[I][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fa[I].s0, fb[j].s0, acc[I][j], 0, 0, 0);
#pragma unroll
    for (int j = 0; j < kFN2; ++j)
      acc[I][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fa[I].s1, fb[j].s1, acc[I][j], 0, 0, 0);
    mfma_i8_rows<I + 1, NB>(acc, fa, fb);
  }
}

// The output tile of 128 WM rows by 256 columns (128 outputs for SwiGLU), a wave
// with its FM x FN accumulators at (wm, wn): scaled and, through LDS as bf16 rows
// (TN columns, the 16-byte chunk of column c of row r at (c / 8) ^ (((r / 4) % 4)
// * 4), so the half-waves' rows r and r + 4 land on different banks), stored in
// 16-byte row stores; 2-byte stores where a row of Y is no whole number of
// vectors.  SX, SW, Y: of the tile's first row and column (Y: row).
template <bool GLU, int FM, int FN, int WM>
__device__ __forceinline__ void store_tile(const i32x16 (&acc)[FM][FN], u32x4 *lds,
                                           const float *__restrict__ SX, const float *__restrict__ SW,
                                           uint16_t *__restrict__ Y, int32_t rows, int32_t wrows,
                                           int32_t n0, int32_t N, int wm, int wn) {
  const int tid = threadIdx.x, lane = tid & 63;
  float sw[FN];
#pragma unroll
  for (int j = 0; j < FN; ++j) {
    const int n = weight_row<GLU>(wn * FN * 32 + j * 32 + (lane & 31));
    sw[j] = SW[n < wrows ? n : wrows - 1];
  }
  const int32_t NO = GLU ? N / 2 : N;
  constexpr int TN = GLU ? kBN2 / 2 : kBN2;
  const bool vec = (NO & 7) == 0;
  const int32_t c0 = GLU ? n0 / 2 : n0;
  uint16_t *so = reinterpret_cast<uint16_t *>(lds);
  float *const ssx = reinterpret_cast<float *>(lds + kBM2 * kBN2 * 2 / 16);
  __syncthreads();   // every wave is done with the slab buffers
  ssx[tid] = SX[tid < rows ? tid : rows - 1];
  __syncthreads();
#define OSW(r_, cv_) ((r_) * TN + (((cv_) ^ ((((r_) >> 2) & 3) << 2)) << 3))
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      const int rr = wm * FM * 32 + i * 32 + (r >> 2) * 8 + (lane >> 5) * 4 + (r & 3);
      const float sx = ssx[rr];
      constexpr int kOut = GLU ? FN / 2 : FN;
#pragma unroll
      for (int j = 0; j < kOut; ++j) {
        float v;
        if constexpr (GLU)
          v = silu_mul((float)acc[i][2 * j][r] * (sx * sw[2 * j]),
                       (float)acc[i][2 * j + 1][r] * (sx * sw[2 * j + 1]));
        else
          v = (float)acc[i][j][r] * (sx * sw[j]);
        const int c = wn * (kOut * 32) + j * 32 + (lane & 31);
        if (vec) so[OSW(rr, c >> 3) + (c & 7)] = bf16_bits(v);
        else if (rr < rows && c0 + c < NO) Y[(int64_t)rr * NO + c0 + c] = bf16_bits(v);
      }
    }
  if (!vec) return;
  __syncthreads();
  constexpr int kVecs = WM * FM * 32 * TN / 8;
#pragma unroll 4
  for (int q = 0; q < kVecs / kGemmThreads; ++q) {
    const int idx = tid + q * kGemmThreads;
    const int rr = idx / (TN / 8), cv = idx % (TN / 8), col = c0 + cv * 8;
    if (rr < rows && col < NO)
      *reinterpret_cast<u32x4 *>(Y + (int64_t)rr * NO + col) =
          *reinterpret_cast<const u32x4 *>(so + OSW(rr, cv));
  }
#undef OSW
}

// A tile of 65 to 128 rows: four waves side by side, each all rows (FM blocks of 32)
// by 64 columns.  X goes through a ring of four slabs that the waves share, a
// barrier each; a wave's columns of W through its own ring of three, read into
// registers at once, so three slabs are on their way and nobody waits for
// another's weights.  256 experts, K = 7168, N = 4096, SwiGLU: 1282 us with 34 rows
// an expert (1630 with 128 x 128 tiles), 1450 with 64 (1660), 1486 with 94 (1710),
// 1790 with 125 (2160); skewed with 64 on average 1034 (1395).  One ring for X and
// W with two slabs in flight: up to 8% more.  At 94 rows it reads 5.6 TB/s (8.3 GB
// with X's misses in L2) and runs 1.2 POP/s together.
constexpr int kHalfRows = 128, kSlabA1 = kHalfRows * kChunks;
template <bool GLU, int FM>
__device__ __forceinline__ void half_tile(__amdgpu_buffer_rsrc_t rX, __amdgpu_buffer_rsrc_t rW,
                                          const float *SX, const float *SW, uint16_t *Y, int32_t rows,
                                          int32_t wrows, int32_t n0, int32_t N, int32_t K, int wv,
                                          u32x4 *lds) {
  constexpr int NA = kSlabA1 / kGemmThreads, NB = kSlabB2 / kGemmThreads;
  static_assert(NA == 4 && NB == 8, "the waits below count 4 loads of X, then 8 of W a slab");
  const int tid = threadIdx.x, lane = tid & 63, l = lane & 31, h = lane >> 5;
  u32x4 *const la = lds, *const lb = lds + 4 * kSlabA1 + wv * (kStreamCols * kChunks);
  uint32_t oa[NA], ob[NB];
#pragma unroll
  for (int i = 0; i < NA; ++i) {
    const int q = i * kGemmThreads + tid, r = q >> 3, c = (q & 7) ^ ((r >> 1) & 7);
    oa[i] = (uint32_t)((r < rows ? r : rows - 1) * K + (K == 64 ? c & 3 : c) * 16);
  }
#pragma unroll
  for (int i = 0; i < NB; ++i) {
    const int r = i * 8 + (lane >> 3), c = (lane & 7) ^ ((r >> 1) & 7);
    const int n = weight_row<GLU>(wv * kStreamCols + r);
    ob[i] = (uint32_t)((n < wrows ? n : wrows - 1) * K + (K == 64 ? c & 3 : c) * 16);
  }
  const int KT = (K + kI8Slab - 1) / kI8Slab;
  const bool half = K % kI8Slab != 0;
  const int last = K > kI8Slab ? K - kI8Slab : 0;
#define LDS_ADDR(p) ((uint32_t)(size_t)LDS_PTR(p))
  const auto issue_x = [&](int kt) {   // into buffer kt % 4
    const int so = kt + 1 < KT ? kt * kI8Slab : last;
#pragma unroll
    for (int i = 0; i < NA; ++i)
      lds_load16(rX, LDS_ADDR(la + (kt & 3) * kSlabA1 + i * kGemmThreads + wv * 64), oa[i], so);
  };
  const auto issue_w = [&](int kt, int buf, int i0, int i1) {
    const int so = kt + 1 < KT ? kt * kI8Slab : last;
#pragma unroll
    for (int i = i0; i < i1; ++i)
      lds_load16_stream(rW, LDS_ADDR(lb + buf * kSlabB2 + i * 64), ob[i], so);
  };
#undef LDS_ADDR
  i32x16 acc[FM][2];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0;
#pragma unroll
  for (int kt = 0; kt < 3; ++kt)
    if (kt < KT) {
      issue_x(kt);
      issue_w(kt, kt, 0, NB);
    }
  int buf = 0;   // of W: kt % 3
  const auto slab = [&](int kt, auto more, auto first) {
    const u32x4 *sa = la + (kt & 3) * kSlabA1, *sb = lb + buf * kSlabB2;
    i32x4 fa[2][FM], fb[4][2];
    constexpr int F = decltype(first)::value;
    const auto read = [&](int c) {
#pragma unroll
      for (int i = 0; i < FM; ++i) fa[c & 1][i] = __builtin_bit_cast(i32x4, sa[swz(i * 32 + l, 2 * c + h)]);
    };
#pragma unroll
    for (int c = F; c < 4; ++c)
#pragma unroll
      for (int j = 0; j < 2; ++j) fb[c][j] = __builtin_bit_cast(i32x4, sb[swz(j * 32 + l, 2 * c + h)]);
    read(F);
#pragma unroll
    for (int c = F; c < 4; ++c) {
      if (c + 1 < 4) read(c + 1);
      if constexpr (decltype(more)::value) {
        if (c == 0) issue_x(kt + 3);
        if (c == 1) asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // W's slab is read: its buffer is free
        if (c > 0) issue_w(kt + 3, buf, c * 3 - 3, c == 3 ? NB : c * 3);
      }
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fa[c & 1][i], fb[c][j], acc[i][j], 0, 0, 0);
    }
    buf = buf == 2 ? 0 : buf + 1;
  };
  // X of slab kt landed for every wave, every wave has read X of slab kt - 1; then
  // this wave's W of slab kt.  Behind them up to two more slabs are on their way.
#define I8H_SYNC(VX, VW)                                                                  \
  asm volatile("s_waitcnt vmcnt(" #VX ") lgkmcnt(0)\n\ts_barrier\n\ts_waitcnt vmcnt(" #VW ")" \
               ::: "memory")
  using std::integral_constant;
  constexpr integral_constant<bool, true> kMore{};
  constexpr integral_constant<bool, false> kNoMore{};
  constexpr integral_constant<int, 0> kWhole{};
  constexpr integral_constant<int, 2> kUpper{};
  int kt = 0;
  for (; kt + 3 < KT; ++kt) {
    I8H_SYNC(32, 24);
    slab(kt, kMore, kWhole);
  }
  if (kt + 2 < KT) {
    I8H_SYNC(32, 24);
    slab(kt, kNoMore, kWhole);
    ++kt;
  }
  if (kt + 1 < KT) {
    I8H_SYNC(20, 12);
    slab(kt, kNoMore, kWhole);
    ++kt;
  }
  I8H_SYNC(8, 0);
  if (half) slab(kt, kNoMore, kUpper);
  else slab(kt, kNoMore, kWhole);
#undef I8H_SYNC
  store_tile<GLU, FM, 2, 1>(acc, lds, SX, SW, Y, rows, wrows, n0, N, 0, wv);
}

template <bool GLU>
__global__ __launch_bounds__(kGemmThreads, 1) void k_grouped_gemm_i8_256(
    const u32x4 *__restrict__ X, const float *__restrict__ SX, const u32x4 *__restrict__ W,
    const float *__restrict__ SW, const u32x4 *__restrict__ Wslot,
    const float *__restrict__ SWslot, const int32_t *__restrict__ tiles,
    const int32_t *__restrict__ ntiles, int32_t max_tiles, int32_t K, int32_t N, int32_t E,
    int32_t n_col_tiles, uint16_t *__restrict__ Y) {
  // two slabs of X and three of W; later the bf16 output tile and the row scales
  __shared__ u32x4 lds[2 * kSlabA2 + 3 * kSlabB2];
  static_assert(kBM2 * kBN2 * 2 + kBM2 * 4 <= (int)sizeof(lds), "output tile and scales fit the buffers");
  static_assert(kBM2 == kGemmThreads, "one row scale per thread");
  u32x4 *const sa = lds, *const sb = lds + 2 * kSlabA2;
  int32_t tile, ctile;
  if (!blocked_tile(ntiles, max_tiles, n_col_tiles, tile, ctile)) return;
  const int32_t n0 = ctile * kBN2;
  const int32_t row0 = tiles[tile * 4 + 0], rows = tiles[tile * 4 + 1], widx = tiles[tile * 4 + 2];
  const int32_t KV = K / 16;
  const bool own = widx < E;
  const int64_t wsel = own ? widx : widx - E;
  const int32_t wrows = N - n0 < kBN2 ? N - n0 : kBN2;
  const float *SWt = (own ? SW : SWslot) + wsel * N + n0;
  // every offset is in range by construction: rows past the end read the last
  // row, and 256 rows of K <= 131071 bytes span less than 2^31
  const __amdgpu_buffer_rsrc_t rX = uniform_rsrc(X + (int64_t)row0 * KV, rows * K);
  const __amdgpu_buffer_rsrc_t rW = uniform_rsrc((own ? W : Wslot) + (wsel * N + n0) * KV, wrows * K);

  const int tid = threadIdx.x, lane = tid & 63;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);  // wave-uniform
  if (rows <= kShortRows) {   // wave wv streams 64 of the 256 columns
    if (n0 + wv * kStreamCols >= N) return;
    const StreamTile t = stream_tile<GLU>(X, SX, (own ? W : Wslot) + wsel * N * KV,
                                          (own ? SW : SWslot) + wsel * N, Y, row0, rows,
                                          n0 + wv * kStreamCols, N, K);
    constexpr int kRing = (2 * kSlabA2 + 3 * kSlabB2) / 4;   // a wave's quarter of LDS
    static_assert(ring_slots(kRingWide) <= kRing, "one wave's ring");
    stream_all<GLU, false, true, false>(t, wv, lane, lds + wv * kRing, nullptr);
    return;
  }
  if (rows <= kHalfRows) {
    static_assert(4 * kSlabA1 + 3 * kSlabB2 <= 2 * kSlabA2 + 3 * kSlabB2, "the rings fit");
    uint16_t *const y = Y + (int64_t)row0 * (GLU ? N / 2 : N);
    if (rows > 96) half_tile<GLU, 4>(rX, rW, SX + row0, SWt, y, rows, wrows, n0, N, K, wv, lds);
    else half_tile<GLU, 3>(rX, rW, SX + row0, SWt, y, rows, wrows, n0, N, K, wv, lds);
    return;
  }
  const int wm = wv >> 1, wn = wv & 1;
  // load i of wave wv fills the 64 slots i*256 + wv*64 + lane, slot q holding
  // chunk (q % 8) ^ ((r / 2) % 8) of LDS row r = q / 8
  uint32_t oa[kLoads2], ob[kLoadsB2];
#pragma unroll
  for (int i = 0; i < kLoads2; ++i) {
    const int q = i * kGemmThreads + tid, r = q >> 3, c = (q & 7) ^ ((r >> 1) & 7);
    oa[i] = (uint32_t)(((r < rows ? r : rows - 1) * KV + (K == 64 ? c & 3 : c)) * 16);
  }
#pragma unroll
  for (int i = 0; i < kLoadsB2; ++i) {
    const int q = i * kGemmThreads + tid, r = q >> 3, c = (q & 7) ^ ((r >> 1) & 7);
    const int n = weight_row<GLU>(r);
    ob[i] = (uint32_t)(((n < wrows ? n : wrows - 1) * KV + (K == 64 ? c & 3 : c)) * 16);
  }
  const int KT = (K + kI8Slab - 1) / kI8Slab;
  const bool half = K % kI8Slab != 0;  // the last slab: only its upper half is new (see k_grouped_gemm_i8)
  const int last = K > kI8Slab ? K - kI8Slab : 0;
#define LDS_ADDR(p) ((uint32_t)(size_t)LDS_PTR(p))
#define I8W_OFF(kt) ((kt) + 1 < KT ? (kt) * kI8Slab : last)
#define I8W_LOAD_X(i, kt, buf)                                                                 \
  lds_load16(rX, LDS_ADDR(&sa[(buf) * kSlabA2 + (i) * kGemmThreads + wv * 64]), oa[i], I8W_OFF(kt));
#define I8W_LOAD_W(i, kt, buf)                                                                 \
  lds_load16(rW, LDS_ADDR(&sb[(buf) * kSlabB2 + (i) * kGemmThreads + wv * 64]), ob[i], I8W_OFF(kt));
#define I8W_ISSUE_X(kt, buf)                                                                   \
  _Pragma("unroll") for (int i = 0; i < kLoads2; ++i) I8W_LOAD_X(i, kt, buf)
#define I8W_ISSUE_W(kt, buf)                                                                   \
  _Pragma("unroll") for (int i = 0; i < kLoadsB2; ++i) I8W_LOAD_W(i, kt, buf)
  static_assert(kLoads2 == 8 && kLoadsB2 == 8, "the waits below count 8 loads of X and 8 of W per slab");
// half h (0 or 1) of a slab: chunks h*4 + lane/32 and h*4 + 2 + lane/32 of the lane's row
#define READ8(FA, FB, bufa, bufb, h, NBK)                                                             \
  {                                                                                            \
    const int c_ = (h) * 4 + (lane >> 5);                                                      \
    _Pragma("unroll") for (int i = 0; i < (NBK); ++i) {                                        \
      const int r_ = wm * kWTM2 + i * 32 + (lane & 31);                                        \
      FA[i].s0 = __builtin_bit_cast(i32x4, sa[(bufa) * kSlabA2 + swz(r_, c_)]);                 \
      FA[i].s1 = __builtin_bit_cast(i32x4, sa[(bufa) * kSlabA2 + swz(r_, c_ + 2)]);             \
    }                                                                                          \
    _Pragma("unroll") for (int j = 0; j < kFN2; ++j) {                                         \
      const int r_ = wn * kWTN2 + j * 32 + (lane & 31);                                        \
      FB[j].s0 = __builtin_bit_cast(i32x4, sb[(bufb) * kSlabB2 + swz(r_, c_)]);                 \
      FB[j].s1 = __builtin_bit_cast(i32x4, sb[(bufb) * kSlabB2 + swz(r_, c_ + 2)]);             \
    }                                                                                          \
  }

  i32x16 acc[kFM2][kFN2];
#pragma unroll
  for (int i = 0; i < kFM2; ++i)
#pragma unroll
    for (int j = 0; j < kFN2; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0;

  Frag2 fa0[kFM2], fb0[kFN2], fa1[kFM2], fb1[kFN2];
  // Each wave waits for its own loads, then the barrier publishes every
  // wave's share; the asm reads one element of each accumulator so that the
  // MFMAs before it stay before it.
#define I8W_SYNC(VM)                                                                           \
  asm volatile("s_waitcnt vmcnt(" #VM ") lgkmcnt(0)\n\ts_barrier"                             \
               :: "a"(acc[0][0][0]), "a"(acc[0][1][0]), "a"(acc[0][2][0]), "a"(acc[0][3][0]),  \
                  "a"(acc[1][0][0]), "a"(acc[1][1][0]), "a"(acc[1][2][0]), "a"(acc[1][3][0]),  \
                  "a"(acc[2][0][0]), "a"(acc[2][1][0]), "a"(acc[2][2][0]), "a"(acc[2][3][0]),  \
                  "a"(acc[3][0][0]), "a"(acc[3][1][0]), "a"(acc[3][2][0]), "a"(acc[3][3][0])   \
               : "memory")
  static_assert(kFM2 == 4 && kFN2 == 4, "the barrier names each of the 16 accumulators");
  // the order of issue is the order the waits count: X0 W0 W1 X1 W2, then X W a slab
  I8W_ISSUE_X(0, 0);
  I8W_ISSUE_W(0, 0);
  if (KT > 1) {
    I8W_ISSUE_W(1, 1);
    I8W_ISSUE_X(1, 1);
  }
  if (KT > 2) {
    I8W_ISSUE_W(2, 2);
    I8W_SYNC(24);   // slab 0 landed
  } else if (KT > 1) {
    I8W_SYNC(16);
  } else {
    I8W_SYNC(0);
  }
#define SGB8(m, n) __builtin_amdgcn_sched_group_barrier(m, n, 0)
// one LDS read after every other MFMA (16 reads, 32 MFMAs)
#define I8W_INTERLEAVE(NBK)                                                                    \
  if constexpr ((NBK) == kFM2) {                                                               \
    _Pragma("unroll") for (int q_ = 0; q_ < 16; ++q_) { SGB8(0x008, 2); SGB8(0x100, 1); }      \
  }
// The second half of a slab: X of slab kt + 2 and W of slab kt + 3 go out.  A
// load occupies the address path for 16 cycles and a wave issues in order: all
// 16 at once would leave the matrix cores idle behind them, so one goes
// between every two MFMAs, with one LDS read (the chunks pinned by
// sched_barrier).
#define I8W_STEP(q_)                                                                           \
  {                                                                                            \
    constexpr int i_ = (q_) / 4, s_ = ((q_) / 2) & 1, j_ = ((q_) & 1) * 2;                     \
    acc[i_][j_] = __builtin_amdgcn_mfma_i32_32x32x32_i8(                                       \
        s_ ? fa1[i_].s1 : fa1[i_].s0, s_ ? fb1[j_].s1 : fb1[j_].s0, acc[i_][j_], 0, 0, 0);     \
    acc[i_][j_ + 1] = __builtin_amdgcn_mfma_i32_32x32x32_i8(                                   \
        s_ ? fa1[i_].s1 : fa1[i_].s0, s_ ? fb1[j_ + 1].s1 : fb1[j_ + 1].s0, acc[i_][j_ + 1],   \
        0, 0, 0);                                                                              \
    /* reads: column fragments first, then the rows' */                                        \
    constexpr int f_ = ((q_) & 7) / 2, h_ = (q_) & 1;                                          \
    const int c_ = (lane >> 5) + 2 * h_;                                                       \
    if constexpr ((q_) < 8) {                                                                  \
      const i32x4 v_ = __builtin_bit_cast(                                                     \
          i32x4, sb[nb * kSlabB2 + swz(wn * kWTN2 + f_ * 32 + (lane & 31), c_)]);              \
      if constexpr (h_ == 0) fb0[f_].s0 = v_; else fb0[f_].s1 = v_;                            \
      I8W_LOAD_X((q_) & 7, kt + 2, ba)                                                         \
    } else {                                                                                   \
      const i32x4 v_ = __builtin_bit_cast(                                                     \
          i32x4, sa[(ba ^ 1) * kSlabA2 + swz(wm * kWTM2 + f_ * 32 + (lane & 31), c_)]);        \
      if constexpr (h_ == 0) fa0[f_].s0 = v_; else fa0[f_].s1 = v_;                            \
      I8W_LOAD_W((q_) & 7, kt + 3, bb)                                                         \
    }                                                                                          \
    __builtin_amdgcn_sched_barrier(0);                                                         \
  }
// slab kt is in buffers ba of X and bb of W, slab kt + 1 in ba ^ 1 and nb; VM: the
// loads that may still be on their way when slab kt + 1 is published
#define I8W_SLAB(NBK, DX, DW, VM)                                                              \
  {                                                                                            \
    const int nb = bb == 2 ? 0 : bb + 1;                                                       \
    READ8(fa1, fb1, ba, bb, 1, NBK);                                                           \
    mfma_i8_rows<0, NBK>(acc, fa0, fb0);                                                       \
    I8W_INTERLEAVE(NBK);                                                                       \
    I8W_SYNC(VM);                                                                              \
    __builtin_amdgcn_sched_barrier(0);                                                         \
    if constexpr ((DX) && (DW) && (NBK) == kFM2) {                                             \
      I8W_STEP(0) I8W_STEP(1) I8W_STEP(2) I8W_STEP(3) I8W_STEP(4) I8W_STEP(5) I8W_STEP(6)      \
      I8W_STEP(7) I8W_STEP(8) I8W_STEP(9) I8W_STEP(10) I8W_STEP(11) I8W_STEP(12) I8W_STEP(13)  \
      I8W_STEP(14) I8W_STEP(15)                                                                \
    } else {                                                                                   \
      if (DX) { I8W_ISSUE_X(kt + 2, ba); }                                                     \
      if (DW) { I8W_ISSUE_W(kt + 3, bb); }                                                     \
      READ8(fa0, fb0, ba ^ 1, nb, 0, NBK);                                                     \
      mfma_i8_rows<0, NBK>(acc, fa1, fb1);                                                     \
      I8W_INTERLEAVE(NBK);                                                                     \
    }                                                                                          \
    ba ^= 1;                                                                                   \
    bb = nb;                                                                                   \
    ++kt;                                                                                      \
  }
// (the last three slabs peeled: fewer loads are on their way)
#define I8W_LOOP(NBK)                                                                          \
  {                                                                                            \
    int kt = 0, ba = 0, bb = 0;                                                                \
    READ8(fa0, fb0, 0, 0, 0, NBK);                                                             \
    while (kt + 3 < KT) I8W_SLAB(NBK, true, true, 8)                                           \
    if (kt + 2 < KT) I8W_SLAB(NBK, true, false, 8)                                             \
    if (kt + 1 < KT) I8W_SLAB(NBK, false, false, 0)                                            \
    READ8(fa1, fb1, ba, bb, 1, NBK);                                                           \
    if (!half) mfma_i8_rows<0, NBK>(acc, fa0, fb0);                                            \
    mfma_i8_rows<0, NBK>(acc, fa1, fb1);                                                       \
  }
  // a wave's 32-row blocks that hold rows: one at least, the tile has more than
  // kHalfRows
  static_assert(kHalfRows >= kWTM2, "both wave rows hold rows of the tile");
  const int live = (rows - wm * kWTM2 + 31) / 32;  // wave-uniform
  if (live >= kFM2) I8W_LOOP(kFM2)
  else if (live == 3) I8W_LOOP(3)
  else if (live == 2) I8W_LOOP(2)
  else I8W_LOOP(1)
#undef I8W_LOOP
#undef I8W_SLAB
#undef I8W_STEP
#undef I8W_INTERLEAVE
#undef SGB8
#undef I8W_SYNC
#undef READ8
#undef I8W_ISSUE_X
#undef I8W_ISSUE_W
#undef I8W_LOAD_X
#undef I8W_LOAD_W
#undef I8W_OFF
#undef LDS_ADDR

  store_tile<GLU, kFM2, kFN2, 2>(acc, lds, SX + row0, SWt, Y + (int64_t)row0 * (GLU ? N / 2 : N), rows,
                                 wrows, n0, N, wm, wn);
}

// Which kernel, by the rows an expert has on average: the streaming kernel while
// groups stay within its one pass of 64 rows over the weights, 256 x 256 tiles
// (whose short tiles stream and whose half tiles take 128 rows) above; 128 x 128
// tiles where N has no 256 columns.  Up to 56 rows where the large tiles are too
// few units for 256 compute units (16 experts, K = 2048, N = 1024, 50 rows: 13.6
// us streaming, 28.8 in large tiles; 64 rows, K = 4096, N = 2048: 77 and 54), up
// to 16 elsewhere: 256 experts, K = 7168, N = 4096, even groups of 19 rows 1167 us
// and 1196, of 32 rows 1256 and 1258, skewed ones of 32 on average 1196 and 749.
// Below: even groups of 4, 8 and 16 rows 1125, 1151, 1174 streaming and 1127, 1145,
// 1155 in large tiles (K = 2048, N = 7168, of 4 and 16: 585, 700 and 612, 638),
// skewed batches of 4, 8 and 16 on average 316, 490, 739 and 323, 421, 530: the
// streaming kernel reads a hot expert's weights once for every 64 of its rows.
enum class I8Kernel { kStream, kTiles, kWide };
static I8Kernel i8_kernel(const Geometry &g, int32_t N) {
  const bool fills = N >= kBN2 && (int64_t)g.E * ((N + kBN2 - 1) / kBN2) >= 256;
  if (g.n <= (int64_t)(fills ? 16 : 56) * g.E) return I8Kernel::kStream;
  return N >= kBN2 ? I8Kernel::kWide : I8Kernel::kTiles;
}
// The streaming kernel splits K while the groups that can have rows, times
// their column tiles, are few units: the GPU holds 2048 of its waves (1536 with
// the larger ring), and a wave by itself takes 48 us for K = 7168 however few
// there are.  K = 7168, two rows an expert, split and not: 20.9 and 48.9 us with
// 256 units, 31.8 and 49.9 with 384, 34.8 and 50.5 with 512, 56.9 and 52.4 with
// 768, 67.8 and 66.2 with 1024.  (K = 2048: 12.3 and 17.4 with 384, 20.2 and 18.2
// with 768; eight rows an expert on 512 units: 19.4 and 19.6.)
constexpr int64_t kStreamWaves = 512;
static bool stream_split(const Geometry &g, int64_t ncol) {
  return (g.n < g.E ? g.n : g.E) * ncol < kStreamWaves;
}
// Small rings (kRingFew) up to this many rows an expert on average (560 us
// against 582 at 4, 403 against 384 at 8).
constexpr int64_t kFewRowsPerExpert = 6;
// ... and goes without the tile table where no group can have many rows (two
// passes over the weights, or a few more where a token names an expert twice):
// the table's launch is most of a small batch's time.
constexpr int32_t kDirectRows = 128;
static bool stream_direct(const Geometry &g, int32_t K) {
  const int32_t most = g.layout == kLL && g.cap < g.T ? g.cap : g.T;
  return most <= kDirectRows && g.n * K <= INT32_MAX;   // 32-bit offsets over a group's rows
}

bool gemm_int8_fits(const Geometry &g, int32_t K, int32_t N) {
  // blocks * threads of a launch stay below 2^32, whichever the tiles
  const int64_t ncol = ((int64_t)N + kStreamCols - 1) / kStreamCols;
  const int64_t most = UINT32_MAX / kGemmThreads;
  return K <= kI8MaxK && gemm_grid_blocks(gemm_max_tiles(g), 1) * ncol <= most &&
         gemm_groups(g) * ncol <= most &&
         blocked_grid(wide_max_tiles(g), ((int64_t)N + kBN2 - 1) / kBN2) <= most;
}

hipError_t launch_grouped_gemm_int8(const Geometry &g, const Workspace &ws, const uint8_t *x,
                                    const float *sx, const uint8_t *w, const float *sw,
                                    const uint8_t *wslot, const float *swslot, int32_t K,
                                    int32_t N, uint16_t *y, bool glu, hipStream_t s) {
  const I8Kernel kind = i8_kernel(g, N);
  const bool wide = kind == I8Kernel::kWide;
  const bool direct = kind == I8Kernel::kStream && stream_direct(g, K);
  const int32_t max_tiles = wide ? wide_max_tiles(g) : gemm_max_tiles(g);
  if (g.n == 0 || max_tiles == 0) return hipSuccess;
  if (!direct) {
    const hipError_t e = launch_gemm_tiles(g, ws, wslot != nullptr, wide ? kShortRows : 0, max_tiles, s);
    if (e != hipSuccess) return e;
  }
  const int32_t cols = wide ? kBN2 : kind == I8Kernel::kStream ? kStreamCols : kBN;
  const int32_t ncol = (N + cols - 1) / cols;
  const TileArgs ta{g, ws, wslot != nullptr ? 1 : 0};
  const bool few = g.n <= kFewRowsPerExpert * g.E;
#define I8_OPERANDS                                                                         \
  reinterpret_cast<const u32x4 *>(x), sx, reinterpret_cast<const u32x4 *>(w), sw,           \
      reinterpret_cast<const u32x4 *>(wslot), swslot
#define I8_LAUNCH(KERN, BLOCKS)                                                             \
  hipLaunchKernelGGL(KERN, dim3((unsigned)(BLOCKS)), dim3(kGemmThreads), 0, s, I8_OPERANDS, \
                     ws.gemm_tiles, ws.gemm_ntiles, max_tiles, K, N, g.E, ncol, y)
#define I8_STREAM1(GLU, FEW, SPLIT, TABLE, BLOCKS)                                          \
  hipLaunchKernelGGL((k_grouped_gemm_i8_stream<GLU, FEW, SPLIT, TABLE>),                    \
                     dim3((unsigned)(BLOCKS)), dim3(SPLIT ? 256 : 64), 0, s, I8_OPERANDS, ta, \
                     max_tiles, K, N, g.E, ncol, y)
#define I8_STREAM(SPLIT, TABLE, BLOCKS)                          \
  do {                                                           \
    if (glu && few) I8_STREAM1(true, true, SPLIT, TABLE, BLOCKS); \
    else if (glu) I8_STREAM1(true, false, SPLIT, TABLE, BLOCKS); \
    else if (few) I8_STREAM1(false, true, SPLIT, TABLE, BLOCKS); \
    else I8_STREAM1(false, false, SPLIT, TABLE, BLOCKS);         \
  } while (0)
  if (wide) {
    if (glu) I8_LAUNCH(k_grouped_gemm_i8_256<true>, blocked_grid(max_tiles, ncol));
    else I8_LAUNCH(k_grouped_gemm_i8_256<false>, blocked_grid(max_tiles, ncol));
  } else if (kind == I8Kernel::kTiles) {
    if (glu) I8_LAUNCH(k_grouped_gemm_i8<true>, gemm_grid_blocks(max_tiles, ncol));
    else I8_LAUNCH(k_grouped_gemm_i8<false>, gemm_grid_blocks(max_tiles, ncol));
  } else if (direct) {
    if (stream_split(g, ncol)) I8_STREAM(true, false, gemm_groups(g) * ncol);
    else I8_STREAM(false, false, gemm_groups(g) * ncol);
  } else {
    if (stream_split(g, ncol)) I8_STREAM(true, true, gemm_grid_blocks(max_tiles, ncol));
    else I8_STREAM(false, true, gemm_grid_blocks(max_tiles, ncol));
  }
#undef I8_STREAM
#undef I8_STREAM1
#undef I8_LAUNCH
#undef I8_OPERANDS
  return hipGetLastError();
}

}  // namespace epk
