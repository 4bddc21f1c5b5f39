// linear_fp8.hip -- matrix product on FP8 operands with a scale per block of 128,
// for the dense half of a layer (shared experts, projections, and their data and
// weight gradients), on gfx950.
//
//   out[m, n] = addend[m, n] + sum_b SX[m, b] * SW[n or n / 128, b] *
//                              sum_{c in block b} X[m, c] * W[n, c]
//
// X is [M, K] e4m3 codes with a scale per row and 128 of K; W is [N, K] with a
// scale per 128 x 128 square (weights) or per row (a gradient's transposed
// operand).  A slab is 128 of K: one scale block, 128 bytes a row.
//
// The weights are the matrix instruction's A operand and the tokens its B
// operand, so a lane's accumulators belong to one token and four consecutive
// channels: with a square's scale (uniform over the wave's channels) the fold of
// a slab's partial sum into the running one is a single fma with a factor per
// lane, and results leave as four channels at a time.
// v_mfma_scale_f32_16x16x128_f8f6f4 takes the whole slab of a 16 x 16 block at
// once, so a partial sum is four registers and two sets of them are enough to
// fold one block while the next is multiplied.
#include <type_traits>

#include "ep_internal.h"
#include "gemm_common.h"

namespace epk {

typedef int i32x8 __attribute__((ext_vector_type(8)));

enum LinearOut : int { kOutBf16 = 0, kOutFp32 = 1, kOutGlu = 2 };

struct LinArgs {
  const u32x4 *x, *w;       // codes, 16-byte vectors
  const float *xs, *ws;
  const void *addend;       // or null
  void *out;
  uint32_t *status;         // or null
  int32_t M, N, K;
};

// silu(g) * u in fp32: the hardware reciprocal and exponential (far below the
// rounding that follows); below -64, where 1 + e^-g leaves the reciprocal's range,
// g * u * e^g in fp64.
__device__ __forceinline__ float silu_times(float g, float u) {
  if (g < -64.0f) return (float)((double)g * (double)u * exp((double)g));
  return g * __builtin_amdgcn_rcpf(1.0f + __expf(-g)) * u;
}

// Channels n .. n + 3 of token m (m < M).  Where rows are not whole vectors each value is a load of
// the addend, which may be the result, and a store behind it: 664 x 1917 x 1536 10.4 us, with an addend
// 12.1, against 7.6 and 7.8 for 1920 channels; 4095 x 2951 x 1280 38 and 62 against 21 and 25 for 2952.
template <int OUT>
__device__ __forceinline__ void store4(const LinArgs &a, int32_t m, int32_t n, f32x4 v) {
  if (n >= a.N) return;
  if constexpr (OUT == kOutGlu) {   // N % 16 == 0: all four are there
    const int64_t at = (int64_t)m * (a.N / 2) + n / 2;
    static_cast<uint32_t *>(a.out)[at / 2] = pack_bf16x2(silu_times(v.x, v.y), silu_times(v.z, v.w));
  } else {
    const int64_t at = (int64_t)m * a.N + n;
    if ((a.N & 3) == 0) {
      if constexpr (OUT == kOutFp32) {
        if (a.addend) v += static_cast<const f32x4 *>(a.addend)[at / 4];
        static_cast<f32x4 *>(a.out)[at / 4] = v;
      } else {
        if (a.addend) {
          const u32x2 r = static_cast<const u32x2 *>(a.addend)[at / 4];
          v += f32x4{bf16_lo(r.x), bf16_hi(r.x), bf16_lo(r.y), bf16_hi(r.y)};
        }
        static_cast<u32x2 *>(a.out)[at / 4] = u32x2{pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w)};
      }
      return;
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      if (n + r >= a.N) break;
      if constexpr (OUT == kOutFp32) {
        static_cast<float *>(a.out)[at + r] = v[r] + (a.addend ? static_cast<const float *>(a.addend)[at + r] : 0.0f);
      } else {
        const float b = a.addend ? bf16_lo(static_cast<const uint16_t *>(a.addend)[at + r]) : 0.0f;
        static_cast<uint16_t *>(a.out)[at + r] = (uint16_t)pack_bf16x2(v[r] + b, 0.0f);
      }
    }
  }
}

// Whether a result's rows are whole 16-byte vectors.
template <int OUT>
__device__ __forceinline__ bool vector_rows(int32_t N) {
  return (N & (OUT == kOutGlu ? 15 : OUT == kOutFp32 ? 3 : 7)) == 0;
}

// Tokens m + (0 .. 15), `live` of them there, x a wave's NA * 16 channels from n, through
// 16 rows of its own in LDS, so that they leave in rows of up to 256 bytes: straight
// from the accumulators a store writes 32 bytes a row, and the tiles of a prefill
// product all end at once.
template <int OUT, int NA>
struct OutBlock {
  static constexpr int channels = NA * (OUT == kOutGlu ? 8 : 16);   // of the result
  static constexpr int stride = channels + 4;                       // floats; rows start four banks apart
  static constexpr int bytes = 16 * stride * 4;
};
template <int OUT, int NA, int MB>
__device__ __forceinline__ void store_block(const LinArgs &a, float *buf, int lane, const f32x4 (&acc)[NA][MB], int j,
                                            int32_t m, int32_t live, int32_t n) {
  using B = OutBlock<OUT, NA>;
  float *const row = buf + (lane & 15) * B::stride;
  const int q = lane >> 4;
#pragma unroll
  for (int i = 0; i < NA; ++i) {
    const f32x4 v = acc[i][j];
    if constexpr (OUT == kOutGlu)
      *reinterpret_cast<f32x2 *>(row + i * 8 + q * 2) = f32x2{silu_times(v.x, v.y), silu_times(v.z, v.w)};
    else
      *reinterpret_cast<f32x4 *>(row + i * 16 + q * 4) = v;
  }
  constexpr int P = OUT == kOutFp32 ? 4 : 8, each = B::channels / P;   // values a piece, pieces a row
  const int32_t N = OUT == kOutGlu ? a.N / 2 : a.N, n0 = OUT == kOutGlu ? n / 2 : n;
#pragma unroll
  for (int t = 0; t < (16 * each + 63) / 64; ++t) {
    const int k = t * 64 + lane, r = k / each, c = (k % each) * P;
    if (r >= 16 || r >= live || n0 + c >= N) continue;
    const f32x4 *const f = reinterpret_cast<const f32x4 *>(buf + r * B::stride + c);
    const int64_t at = ((int64_t)(m + r) * N + n0 + c) / P;
    if constexpr (OUT == kOutFp32) {
      f32x4 v = f[0];
      if (a.addend) v += static_cast<const f32x4 *>(a.addend)[at];
      static_cast<f32x4 *>(a.out)[at] = v;
    } else {
      float v[8] = {f[0].x, f[0].y, f[0].z, f[0].w, f[1].x, f[1].y, f[1].z, f[1].w};
      if (OUT == kOutBf16 && a.addend) {
        float r8[8];
        unpack8(static_cast<const u32x4 *>(a.addend)[at], r8);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] += r8[e];
      }
      static_cast<u32x4 *>(a.out)[at] = pack8(v);
    }
  }
}

__device__ __forceinline__ i32x8 join_codes(const u32x4 lo, const u32x4 hi) {
  return i32x8{(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
}
__device__ __forceinline__ f32x4 mfma_slab(const i32x8 &a, const i32x8 &b, const f32x4 &c) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 0, 0, 0, 127, 0, 127);  // both e4m3, times 2^0
}

// Codes 8 g .. 8 g + 7 of a lane's 32 of a slab, times 2^(exponent of s), as a bf16
// operand: exact.
__device__ __forceinline__ bf16x8 widen(const i32x8 &c, int g, float s) {
  bf16x8 o;
#pragma unroll
  for (int h = 0; h < 4; ++h) {
    const uint32_t w = (uint32_t)c[2 * g + (h >> 1)];
    const bf16x2 v = (h & 1) ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, s, true)
                             : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, s, false);
    o[2 * h] = v.x;
    o[2 * h + 1] = v.y;
  }
  return o;
}
__device__ __forceinline__ int exponent_of(float s) { return (int)((__float_as_uint(s) >> 23) & 0xFFu); }

// Scales a caller called powers of two: if one is not, the flag goes into *status.
// The workgroup's threads share the n scales.
__device__ __forceinline__ void check_scales(const float *s, int64_t n, uint32_t *status) {
  uint32_t bad = 0u;
  for (int64_t i = threadIdx.x; i < n; i += blockDim.x) (void)scale_exponent(s[i], &bad);
  if (__ballot(bad != 0u) != 0u && (threadIdx.x & 63) == 0) atomicOr(status, kFlagScaleFormat);
}
#define LDS_ADDR(p) ((uint32_t)(size_t)LDS_PTR(p))

// ---------------------------------------------------------------------------
// tiles
//
// WN x WM waves, each NA x MB blocks of 16 channels x 16 tokens.  Slabs go from
// global memory straight into LDS, ST buffers of them: slab k + ST is sent for once
// slab k has been read, so it has ST - 1 slabs' products to land in.  Two slabs of the
// large tiles fill LDS; the smallest, which wait for memory, hold four.
//
// fp32 results (a main gradient) want every product whole: the FP8 instruction cuts
// the products of 8 neighbouring k at 2^-13 of the largest one's binade, which a bf16
// result does not show and an fp32 one does.  Their operands are widened to bf16,
// which is exact, at half the instruction's rate.  Power-of-two scales go into the
// instruction's (or the widening's) exponents and leave nothing to fold.
//
// 4096 x 4096 x 7168: 109 us with amax scales (2.2 PFLOP/s), 97 with powers of two,
// 192 and 174 with fp32 results; 8192^3 450 and 421 (2.45 and 2.6).  Of the large
// tiles' time the matrix cores are busy half: loads into LDS, reads out of it and the
// fold of the sums interleave with the products and are none of them the bound alone
// (without the loads 94 us, without the reads 98).  Small tiles wait for their
// operands, which were measured to reach a compute unit at 65 to 70 GB/s.

template <int WN_, int WM_, int NA_, int MB_, int ST_>
struct LinShape {
  static constexpr int WN = WN_, WM = WM_, NA = NA_, MB = MB_, ST = ST_;   // ST: slabs in LDS
  static constexpr int BN = WN * NA * 16, BM = WM * MB * 16, threads = 64 * WN * WM;
};

// Tile of workgroup blockIdx.x: XCD x (b % 8) takes a contiguous eighth of the
// tiles, in blocks of `span` token tiles by all channel tiles, tokens first, so
// that the tiles an XCD runs at once share their rows and weights in its L2.
__device__ __forceinline__ bool linear_tile(int32_t tm, int32_t tn, int32_t span, int32_t &mt, int32_t &nt) {
  const int32_t total = tm * tn, per = (total + kXcds - 1) / kXcds;
  const int32_t x = blockIdx.x % kXcds, slot = blockIdx.x / kXcds, i = x * per + slot;
  if (slot >= per || i >= total) return false;
  const int32_t g = i / (span * tn), rem = i - g * span * tn;
  const int32_t h = tm - g * span < span ? tm - g * span : span;
  mt = g * span + rem % h;
  nt = rem / h;
  return true;
}

template <class S, bool ROW, bool POW2, int OUT>
__global__ __launch_bounds__(S::threads, 2) void k_linear_fp8(LinArgs a, int32_t tm, int32_t tn,
                                                              int32_t span) {
  constexpr bool EXACT = OUT == kOutFp32;
  constexpr int NA = S::NA, MB = S::MB;
  // rows whose scales a tile reads: its tokens', then its channels' or its squares'
  constexpr int NS = S::BM + (ROW ? S::BN : 64);
  constexpr int kSlabW = S::BN * kChunks, kSlabX = S::BM * kChunks;
  __shared__ u32x4 slabs[S::ST * (kSlabW + kSlabX)];   // of weights, then of tokens; in the end the results
  u32x4 *const sw = slabs, *const sx = slabs + S::ST * kSlabW;
  // Four slabs' scales a buffer.  Those of the four after are under way beside them; slab
  // kt + ST goes out when slab kt + 1 is next to be read, whose four lie one buffer back
  // with ST 2, up to two with ST 4.
  constexpr int SB = S::ST == 2 ? 2 : 4;
  static_assert(S::ST == 2 || S::ST == 4, "slabs in LDS");
  __shared__ __attribute__((aligned(16))) float ssc[SB][NS][4];
  int32_t mt, nt;
  if (!linear_tile(tm, tn, span, mt, nt)) return;
  const int32_t m0 = mt * S::BM, n0 = nt * S::BN;
  const int32_t rows = a.M - m0 < S::BM ? a.M - m0 : S::BM, wrows = a.N - n0 < S::BN ? a.N - n0 : S::BN;
  const int32_t KV = a.K / 16, NB = a.K / 128;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);   // wave-uniform
  const int wn = wv / S::WM, wm = wv % S::WM;

  // resources over the tile's rows (32-bit offsets: K <= 2^22); rows past the end are out of their
  // range, by the lane's offset alone, and read as zeros
  const __amdgpu_buffer_rsrc_t rW = __builtin_amdgcn_make_buffer_rsrc(
      (void *)(a.w + (int64_t)n0 * KV), (short)0, wrows * a.K, kBufDword3);
  const __amdgpu_buffer_rsrc_t rX = __builtin_amdgcn_make_buffer_rsrc(
      (void *)(a.x + (int64_t)m0 * KV), (short)0, rows * a.K, kBufDword3);
  constexpr int LW = S::BN * kChunks / S::threads, LX = S::BM * kChunks / S::threads;
  static_assert(LW * S::threads == S::BN * kChunks && LX * S::threads == S::BM * kChunks, "whole loads");
  // Slot q of a slab holds chunk (q % 8) ^ ((r / 2) % 8) of row r = q / 8.  A load of
  // the workgroup fills kStep rows (a multiple of 16: the same chunk in each).
  constexpr int kStep = S::threads / 8;
  static_assert(kStep % 16 == 0, "the swizzle repeats");
  const uint32_t off = (uint32_t)(((tid >> 3) * KV + ((tid & 7) ^ ((tid >> 4) & 7))) * 16);
  // Scales travel four slabs at a time, since a row's lie next to each other (16
  // lines a load, where one slab's scales of 64 rows are 64): with slab k go the
  // scales of rows 16 ((k + 3) % 4) .. + 15 of each 64 for slabs 4 g .. 4 g + 3, g =
  // (k + 3) / 4, so that they are whole with slab 4 g.  Each wave brings 64 rows'
  // (some the same ones as another).
  static_assert(NS / 64 <= S::WN * S::WM, "a load of scales a wave");
  const int32_t nsq = (a.N + 127) / 128;
  const int part = wv % (NS / 64);
  const bool of_x = part < S::BM / 64;   // wave-uniform
  const int32_t first = of_x ? 0 : ROW ? n0 : n0 / 128, left = (of_x ? rows : ROW ? wrows : nsq - first);
  const uint32_t osc = (uint32_t)((((of_x ? part : part - S::BM / 64) * 64 + (lane >> 2)) * NB + (lane & 3)) * 4);
  const __amdgpu_buffer_rsrc_t rS = __builtin_amdgcn_make_buffer_rsrc(
      (void *)(of_x ? a.xs + (int64_t)m0 * NB : a.ws + (int64_t)first * NB), (short)0,
      (left < 512 ? left : 512) * NB * 4, kBufDword3);
  // rows past the end, slabs past the last: unused.  The whole offset is the lane's: what lies past the
  // last row's last slab is out of the resource's range
  const auto issue_scales = [&](int32_t four, int piece) {
    lds_load4(rS, LDS_ADDR(&ssc[four & (SB - 1)][part * 64 + piece * 16][0]), osc + (uint32_t)(piece * 64 * NB + four * 16), 0);
  };
  static_assert(128 % (NA * 16) == 0 && NA % 2 == 0, "a wave's channels lie in one square");
  constexpr int kLoads = LW + LX + 1;   // of a wave, a slab
  // loads lo .. hi - 1 of slab k's kLoads
  const auto issue = [&](int32_t k, int buf, int lo, int hi) {
    const int32_t kt = k < NB ? k : NB - 1;   // past the end: the last slab again, which nobody reads
#pragma unroll
    for (int i = lo; i < hi; ++i) {
      if (i < LX) lds_load16(rX, LDS_ADDR(&sx[buf * kSlabX + i * S::threads + wv * 64]), off + (uint32_t)(i * kStep * a.K), kt * 128);
      else if (i < LX + LW)
        lds_load16(rW, LDS_ADDR(&sw[buf * kSlabW + (i - LX) * S::threads + wv * 64]), off + (uint32_t)((i - LX) * kStep * a.K), kt * 128);
      else issue_scales((k + 3) >> 2, (k + 3) & 3);
    }
  };
  // a lane's 32 codes of a slab are chunks q and q + 4 of its row, q = lane / 16 (the same for both
  // operands, which is all the product needs): the 16 lanes that LDS serves at a time -- 0-3, 12-15,
  // 20-27, then 4-11, 16-19, 28-31 -- then meet 16 different places of its 256-byte rows, where
  // chunks 2 q and 2 q + 1 met every one twice
  const int rl = lane & 15, cl = lane >> 4;

  f32x4 acc[NA][MB];
#pragma unroll
  for (int i = 0; i < NA; ++i)
#pragma unroll
    for (int j = 0; j < MB; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  // weight fragments, read two steps ahead (one where registers run out)
  constexpr int WD = NA == 8 && (POW2 || ROW) ? 2 : 3;
  static_assert(!EXACT || WD == 3, "the next step's fragment is widened under this step's products");
  i32x8 wf[WD];
  float wsc[WD];     // row scales with POW2: those of the fragments' rows
  f32x4 sn[4], sl;   // ... without: of the lane's four channels in the fragments; in the slab's last one
  f32x4 p[MB];       // the last step's partial sums, folded under the next step's products
  i32x8 xf[MB];      // the wave's token fragments
  bf16x8 xb[EXACT ? MB : 1][4], wb[2];   // EXACT: the widened ones, and two chunks of a weight fragment
  float sa[MB], sb[MB], qa = 1.0f, qb = 1.0f;   // their scales and the square's, two slabs in turn
#pragma unroll
  for (int j = 0; j < MB; ++j) {
    p[j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    sb[j] = 0.0f;
  }
  sl = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  const auto read_w = [&](int buf, int32_t k, int i) {
    const int r = (wn * NA + i) * 16 + rl;
    wf[i % WD] = join_codes(sw[buf * kSlabW + swz(r, cl)], sw[buf * kSlabW + swz(r, cl + 4)]);
    if constexpr (POW2 && ROW) wsc[i % WD] = ssc[(k >> 2) & (SB - 1)][S::BM + r][k & 3];
    if constexpr (!POW2 && ROW) {
#pragma unroll
      for (int q = 0; q < 4; ++q)
        sn[i & 3][q] = ssc[(k >> 2) & (SB - 1)][S::BM + (wn * NA + i) * 16 + (lane >> 4) * 4 + q][k & 3];
    }
  };
  const auto read_x = [&](int buf, int j) {
    const int r = (wm * MB + j) * 16 + rl;
    xf[j] = join_codes(sx[buf * kSlabX + swz(r, cl)], sx[buf * kSlabX + swz(r, cl + 4)]);
  };
  const auto read_s = [&](int32_t k, float (&f)[MB], float &q) {
    q = ROW ? 1.0f : ssc[(k >> 2) & (SB - 1)][ROW ? 0 : S::BM + wn * NA * 16 / 128][k & 3];
#pragma unroll
    for (int j = 0; j < MB; ++j) f[j] = ssc[(k >> 2) & (SB - 1)][(wm * MB + j) * 16 + rl][k & 3];
  };
  const auto fold = [&](int i, int j, float f, const f32x4 &n) {
#pragma unroll
    for (int q = 0; q < 4; ++q) acc[i][j][q] = __builtin_fmaf(p[j][q], ROW ? n[q] * f : f, acc[i][j][q]);
  };
  // A slab whose token fragments, first two weight fragments and scales f, fq are
  // in registers.  Before its last step everyone's reads of it are done and the
  // next slab has landed: the next slab's first fragments are read, a token fragment
  // as soon as the last products that use its registers are under way, and slab
  // kt + ST is sent for, into this one's place, LP loads behind each product from
  // there on into the next slab (all at once they hold up the products behind
  // them).  A step's sums are folded under the next step's products (the last one's
  // under the next slab's first, with that slab's scales g, which the next slab's
  // replace only then).  sched_barrier holds that order: left alone, the compiler
  // folds each sum at once and waits for it.
  constexpr int LP = (kLoads + NA * MB - 1) / (NA * MB);
  constexpr int kFirst = MB * LP < kLoads ? MB * LP : kLoads;   // a slab's loads under the last step
  const auto slab = [&](int32_t kt, int buf, int nbuf, float (&f)[MB], float &fq, float (&g)[MB], float &gq) {
    if constexpr (!ROW && !POW2) {
#pragma unroll
      for (int j = 0; j < MB; ++j) f[j] *= fq;
    }
    int ex[MB], eq = 127;
    if constexpr (POW2 && !EXACT) {
#pragma unroll
      for (int j = 0; j < MB; ++j) ex[j] = exponent_of(f[j]);
      if constexpr (!ROW) eq = exponent_of(fq);
    }
#pragma unroll
    for (int i = 0; i < NA; ++i) {
      const bool last = i + 1 == NA;
      const i32x8 w = wf[i % WD];
      const float ws = POW2 && ROW ? wsc[i % WD] : fq;
      const f32x4 n = i > 0 ? sn[(i - 1) & 3] : sl;
      if (i + WD - 1 < NA) read_w(buf, kt, i + WD - 1);
      if (last) {
        if constexpr (ROW && !POW2) sl = sn[i & 3];
        asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"((S::ST - 2) * kLoads) : "memory");
        __builtin_amdgcn_sched_barrier(0);
        read_w(nbuf, kt + 1, 0);
        if constexpr (WD == 3) read_w(nbuf, kt + 1, 1);
        read_s(kt + 1, g, gq);
      }
      // what goes out behind product j: loads at .. at + LP - 1 of slab kt + ST in the
      // last step, of slab kt - 1 + ST before
      const auto behind = [&](int j) {
        if (last) read_x(nbuf, j);
        const int at = (last ? j : (i + 1) * MB + j) * LP;
        issue(last ? kt + S::ST : kt - 1 + S::ST, last ? buf : (S::ST == 2 ? nbuf : (kt - 1) & (S::ST - 1)), at,
              at + LP < kLoads ? at + LP : kLoads);
        __builtin_amdgcn_sched_barrier(0);
      };
      if constexpr (EXACT) {
        // chunk c's products, and under them the next chunk's widening: of the weights, and
        // in the first step of the tokens (the next slab's in the last)
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int j = 0; j < MB; ++j) {
            f32x4 &t = POW2 ? acc[i][j] : p[j];
            if (!POW2 && c == 0) fold(i > 0 ? i - 1 : NA - 1, j, i > 0 ? f[j] : g[j], n);
            t = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wb[c & 1], xb[j][c],
                                                        !POW2 && c == 0 ? f32x4{0.0f, 0.0f, 0.0f, 0.0f} : t, 0, 0, 0);
            if (c == 0) behind(j);
            if (i == 0 && c < 3) xb[j][c + 1] = widen(xf[j], c + 1, POW2 ? f[j] : 1.0f);
            if (last && c == 3) xb[j][0] = widen(xf[j], 0, POW2 ? g[j] : 1.0f);
            if (j == 0) {
              if (c < 3) wb[(c + 1) & 1] = widen(w, c + 1, POW2 ? ws : 1.0f);
              else wb[0] = widen(wf[last ? 0 : (i + 1) % WD], 0, !POW2 ? 1.0f : ROW ? wsc[last ? 0 : (i + 1) % WD] : last ? gq : fq);
            }
            __builtin_amdgcn_sched_barrier(0);
          }
      } else if constexpr (POW2) {
        const int ew = ROW ? exponent_of(ws) : eq;
#pragma unroll
        for (int j = 0; j < MB; ++j) {
          acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, xf[j], acc[i][j], 0, 0, 0, ew, 0, ex[j]);
          behind(j);
        }
      } else {
#pragma unroll
        for (int j = 0; j < MB; ++j) {
          fold(i > 0 ? i - 1 : NA - 1, j, i > 0 ? f[j] : g[j], n);
          p[j] = mfma_slab(w, xf[j], f32x4{0.0f, 0.0f, 0.0f, 0.0f});
          behind(j);
        }
      }
    }
  };
#pragma unroll
  for (int i = 0; i < 4; ++i) issue_scales(0, i);
#pragma unroll
  for (int i = 0; i < S::ST; ++i) issue(i, i, 0, i + 1 < S::ST ? kLoads : kFirst);
  asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"((S::ST - 2) * kLoads + kFirst) : "memory");   // slab 0 landed
#pragma unroll
  for (int j = 0; j < MB; ++j) read_x(0, j);
  read_s(0, sa, qa);
  read_w(0, 0, 0);
  if constexpr (WD == 3) read_w(0, 0, 1);
  if constexpr (EXACT) {
#pragma unroll
    for (int j = 0; j < MB; ++j) xb[j][0] = widen(xf[j], 0, POW2 ? sa[j] : 1.0f);
    wb[0] = widen(wf[0], 0, !POW2 ? 1.0f : ROW ? wsc[0] : qa);
  }
  static_assert((S::ST & (S::ST - 1)) == 0 && S::ST >= 2, "slab kt is in buffer kt % ST");
  constexpr int kMask = S::ST - 1;
  int32_t kt = 0;
  for (; kt + 1 < NB; kt += 2) {
    const int b = S::ST == 2 ? 0 : kt & kMask;   // (kt is even)
    slab(kt, b, b + 1, sa, qa, sb, qb);
    slab(kt + 1, b + 1, S::ST == 2 ? 0 : (kt + 2) & kMask, sb, qb, sa, qa);
  }
  if (kt < NB) {
    const int b = S::ST == 2 ? 0 : kt & kMask;
    slab(kt, b, b + 1, sa, qa, sb, qb);
#pragma unroll
    for (int j = 0; j < MB; ++j) sb[j] = sa[j];
  }
  if constexpr (!POW2) {
#pragma unroll
    for (int j = 0; j < MB; ++j) fold(NA - 1, j, sb[j], sl);
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // nothing lands after the workgroup has ended
  if constexpr (POW2) {
    if (a.status) {   // each scale by one workgroup
      if (nt == 0) check_scales(a.xs + (int64_t)m0 * NB, (int64_t)rows * NB, a.status);
      if (mt == 0 && ROW) check_scales(a.ws + (int64_t)n0 * NB, (int64_t)wrows * NB, a.status);
      if (mt == 0 && !ROW && n0 % 128 == 0)
        check_scales(a.ws + (int64_t)(n0 / 128) * NB, (int64_t)((wrows + 127) / 128) * NB, a.status);
    }
  }
  if (vector_rows<OUT>(a.N)) {
    static_assert(S::WN * S::WM * OutBlock<OUT, NA>::bytes <= (int)sizeof(slabs), "the waves' rows fit");
    __syncthreads();   // every wave is done with the slabs
    float *const buf = reinterpret_cast<float *>(slabs) + wv * (OutBlock<OUT, NA>::bytes / 4);
#pragma unroll
    for (int j = 0; j < MB; ++j) {
      const int32_t m = (wm * MB + j) * 16;
      store_block<OUT>(a, buf, lane, acc, j, m0 + m, rows - m, n0 + wn * NA * 16);
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < MB; ++j) {
    const int32_t m = (wm * MB + j) * 16 + rl;
    if (m >= rows) continue;
#pragma unroll
    for (int i = 0; i < NA; ++i)
      store4<OUT>(a, m0 + m, n0 + (wn * NA + i) * 16 + (lane >> 4) * 4, acc[i][j]);
  }
}

// ---------------------------------------------------------------------------
// few tokens
//
// A workgroup takes 16 NC channels and 16 MT tokens, its waves every so many slabs each:
// the weights are streamed once where that is all the tokens.  A wave keeps a ring of slabs
// in LDS of its own -- no barrier until the end -- filled by loads whose lanes
// follow the memory: in the matrix instruction's order consecutive lanes are rows
// apart and a load of 1 KB holds the address unit 88 cycles where it takes 22 (16
// tokens, N 4096, K 7168: 11.0 us, straight into registers).  The waves' sums are
// joined through LDS in a fixed order.

template <int MT>
struct FewShape {
  static constexpr int waves = MT == 4 ? 4 : 8, ring = MT == 1 ? 4 : 3;   // LDS: 147, 160, 129 (153) KB
};

template <int MT, int NC, bool ROW, bool POW2, int OUT>
__global__ __launch_bounds__(64 * FewShape<MT>::waves) void k_linear_fp8_few(LinArgs a) {
  constexpr int W = FewShape<MT>::waves, R = FewShape<MT>::ring, BN = NC * 16;
  __shared__ u32x4 slabs[W][R][(NC + MT) * 16 * kChunks];   // the rows of weights, then the tokens
  __shared__ float scales[W][R][128];                      // the tokens', then the channels' or the square's
  const int tid = threadIdx.x, lane = tid & 63, rl = lane & 15, q4 = lane >> 4;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int32_t n0 = blockIdx.x * BN, m0 = blockIdx.y * MT * 16, NB = a.K / 128;
  const int32_t rows = a.M - m0 < MT * 16 ? a.M - m0 : MT * 16, wrows = a.N - n0 < BN ? a.N - n0 : BN;
  const __amdgpu_buffer_rsrc_t rW = __builtin_amdgcn_make_buffer_rsrc(
      (void *)(a.w + (int64_t)n0 * (a.K / 16)), (short)0, wrows * a.K, kBufDword3);
  const __amdgpu_buffer_rsrc_t rX = __builtin_amdgcn_make_buffer_rsrc(
      (void *)(a.x + (int64_t)m0 * (a.K / 16)), (short)0, rows * a.K, kBufDword3);
  const __amdgpu_buffer_rsrc_t rXS = __builtin_amdgcn_make_buffer_rsrc(
      (void *)(a.xs + (int64_t)m0 * NB), (short)0, rows * NB * 4, kBufDword3);
  const __amdgpu_buffer_rsrc_t rWS = __builtin_amdgcn_make_buffer_rsrc(
      (void *)(a.ws + (int64_t)(ROW ? n0 : n0 / 128) * NB), (short)0, (ROW ? wrows : 1) * NB * 4, kBufDword3);
  // eight rows a load, chunks in the order of swz; rows past the end are out of range
  const uint32_t off = (uint32_t)((lane >> 3) * a.K + ((lane & 7) ^ ((lane >> 4) & 3)) * 16);
  const uint32_t oxs = (uint32_t)((lane < rows ? lane : rows - 1) * NB * 4);
  const int32_t cw = lane & (BN - 1);
  const uint32_t ows = ROW ? (uint32_t)((cw < wrows ? cw : wrows - 1) * NB * 4) : 0u;
  constexpr int kLoads = 2 * NC + 2 * MT + 2;
  const auto issue = [&](int32_t k, int slot) {
    u32x4 *const d = slabs[wv][slot];
#pragma unroll
    for (int i = 0; i < 2 * NC; ++i)   // rows 8 i ..: every second eight's chunks are permuted by 4 more
      lds_load16_stream(rW, LDS_ADDR(d + i * 64), (off ^ (uint32_t)((i & 1) * 64)) + (uint32_t)(i * 8 * a.K), k * 128);
#pragma unroll
    for (int i = 0; i < 2 * MT; ++i)
      lds_load16(rX, LDS_ADDR(d + (2 * NC + i) * 64), (off ^ (uint32_t)((i & 1) * 64)) + (uint32_t)(i * 8 * a.K), k * 128);
    lds_load4(rXS, LDS_ADDR(&scales[wv][slot][0]), oxs, k * 4);
    lds_load4(rWS, LDS_ADDR(&scales[wv][slot][64]), ows, k * 4);
  };
  f32x4 acc[NC][MT];
#pragma unroll
  for (int c = 0; c < NC; ++c)
#pragma unroll
    for (int j = 0; j < MT; ++j) acc[c][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  // slab in `slot`, landed; `next`, if it is one, is sent for into its place once it is read
  const auto slab = [&](int slot, int32_t next) {
    const u32x4 *const d = slabs[wv][slot];
    const float *const sc = scales[wv][slot];
    i32x8 fw[NC], fx[MT];
    float s[MT], sw[NC];
    f32x4 sn[NC];
#pragma unroll
    for (int c = 0; c < NC; ++c) fw[c] = join_codes(d[swz(c * 16 + rl, q4)], d[swz(c * 16 + rl, q4 + 4)]);
#pragma unroll
    for (int j = 0; j < MT; ++j) {
      fx[j] = join_codes(d[swz((NC + j) * 16 + rl, q4)], d[swz((NC + j) * 16 + rl, q4 + 4)]);
      s[j] = sc[j * 16 + rl];
    }
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      if constexpr (POW2) {   // of the fragment's row
        sw[c] = sc[64 + (ROW ? c * 16 + rl : 0)];
      } else {                // of the result's channels
#pragma unroll
        for (int r = 0; r < 4; ++r) sn[c][r] = sc[64 + (ROW ? c * 16 + q4 * 4 + r : 0)];
      }
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    if (next < NB) issue(next, slot);
    // powers of two go into the operands' exponents, as in the tiles: the product of two may lie outside
    // fp32 where the result does not
#pragma unroll
    for (int c = 0; c < NC; ++c) {
#pragma unroll
      for (int j = 0; j < MT; ++j) {
        f32x4 p = POW2 ? acc[c][j] : f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        if constexpr (OUT == kOutFp32) {
#pragma unroll
          for (int g = 0; g < 4; ++g)
            p = __builtin_amdgcn_mfma_f32_16x16x32_bf16(widen(fw[c], g, POW2 ? sw[c] : 1.0f),
                                                        widen(fx[j], g, POW2 ? s[j] : 1.0f), p, 0, 0, 0);
        } else if constexpr (POW2) {
          p = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fw[c], fx[j], p, 0, 0, 0, exponent_of(sw[c]), 0,
                                                               exponent_of(s[j]));
        } else {
          p = mfma_slab(fw[c], fx[j], p);
        }
        if constexpr (POW2) {
          acc[c][j] = p;
        } else {
#pragma unroll
          for (int r = 0; r < 4; ++r) acc[c][j][r] = __builtin_fmaf(p[r], sn[c][r] * s[j], acc[c][j][r]);
        }
      }
    }
  };
  int32_t k = wv;
#pragma unroll
  for (int i = 0; i < R; ++i)
    if (k + i * W < NB) issue(k + i * W, i);
  int slot = 0;
  for (; k + (R - 1) * W < NB; k += W) {   // R slabs under way: the first has landed
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"((R - 1) * kLoads) : "memory");
    slab(slot, k + R * W);
    slot = slot + 1 == R ? 0 : slot + 1;
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  for (; k < NB; k += W) {
    slab(slot, NB);
    slot = slot + 1 == R ? 0 : slot + 1;
  }
  if constexpr (POW2) {
    if (a.status) {
      if (blockIdx.x == 0) check_scales(a.xs + (int64_t)m0 * NB, (int64_t)rows * NB, a.status);
      if (ROW || n0 % 128 == 0)
        check_scales(a.ws + (int64_t)(ROW ? n0 : n0 / 128) * NB, (int64_t)(ROW ? wrows : 1) * NB, a.status);
    }
  }
  f32x4 *const red = reinterpret_cast<f32x4 *>(&slabs[0][0][0]);
  static_assert(W * NC * MT * 64 * 16 <= (int)sizeof(slabs), "the waves' sums fit");
  __syncthreads();
#pragma unroll
  for (int c = 0; c < NC; ++c)
#pragma unroll
    for (int j = 0; j < MT; ++j) red[((wv * NC + c) * MT + j) * 64 + lane] = acc[c][j];
  __syncthreads();
  for (int e = tid; e < NC * MT * 64; e += 64 * W) {
    f32x4 v = red[e];
#pragma unroll
    for (int i = 1; i < W; ++i) v += red[i * NC * MT * 64 + e];
    const int32_t b = e >> 6, m = m0 + (b % MT) * 16 + (e & 15);
    if (m < a.M) store4<OUT>(a, m, n0 + (b / MT) * 16 + ((e >> 4) & 3) * 4, v);
  }
}

// ---------------------------------------------------------------------------

typedef LinShape<2, 4, 8, 4, 2> Shape256;      // 256 x 256, 8 waves of 128 x 64
typedef LinShape<2, 4, 4, 3, 2> Shape128x192;  // 128 channels x 192 tokens, 8 waves of 64 x 48
typedef LinShape<2, 2, 4, 4, 2> Shape128;      // 128 x 128, 4 waves of 64 x 64
typedef LinShape<2, 2, 2, 2, 4> Shape64;       // 64 x 64, 4 waves of 32 x 32

// Time of a compute unit's share of the tiles, in us: a tile alone on it takes `one`
// a slab and `more` besides (prologue, results), two side by side `two` and `more2`
// (0: two do not fit).  Measured with 256, 512, 768 and 1024 tiles at K 2048 and
// 6144, shared by all forms of the scales.
struct TileTimes {
  double one, more, two, more2;
};
template <class S>
static double tiles_time(const Linear &n, const TileTimes &t) {
  const int64_t tiles = (int64_t)((n.M + S::BM - 1) / S::BM) * ((n.N + S::BN - 1) / S::BN);
  const int64_t each = (tiles + 255) / 256, pairs = t.two > 0.0 ? each / 2 : 0;
  const double slabs = n.K / 128;
  return (double)pairs * (t.two * slabs + t.more2) + (double)(each - 2 * pairs) * (t.one * slabs + t.more);
}
static int64_t tiles_of(const Linear &n, int32_t b) {
  return (int64_t)((n.M + b - 1) / b) * ((n.N + b - 1) / b);
}

template <class S, bool ROW, bool POW2, int OUT>
static void launch_tiles(const LinArgs &a, int32_t span, hipStream_t s) {
  const int32_t tm = (a.M + S::BM - 1) / S::BM, tn = (a.N + S::BN - 1) / S::BN;
  const unsigned grid = (unsigned)((((int64_t)tm * tn + kXcds - 1) / kXcds) * kXcds);
  hipLaunchKernelGGL((k_linear_fp8<S, ROW, POW2, OUT>), dim3(grid), dim3(S::threads), 0, s, a, tm, tn, span);
}

// Blocks of 16 tokens and of 16 channels a workgroup of the kernel for few tokens takes, or no tokens for
// tiles: as few as keep its workgroups, whose waves share K, to one a compute unit (128 x 1024 x 7168 8.0
// us, fp32 results 8.3, against 16.8 and 26.4 with 64 x 64 tiles), and up to 32 tokens whatever the
// channels.  64 tokens and 32 channels, whose slabs are as long in coming as a tile's, only where their
// widening is shared by the waves or K is short (256 x 2048 x 7168 with fp32 results 18.0 against 26.7,
// in bf16 17.0 both, 64 x 8192 x 7168 19.4 against 17.1; 256 x 2048 x 1024 4.2 against 5.0).  K 0 leaves
// the addend, or zeros.
struct FewBlocks {
  int mt, nc;
  int64_t channels(const Linear &n) const { return ((int64_t)n.N + 16 * nc - 1) / (16 * nc); }
  int64_t tokens(const Linear &n) const { return (n.M + 16 * mt - 1) / (16 * mt); }
};
static FewBlocks few_blocks(const Linear &n) {
  if (n.K == 0) return {4, 1};
  for (const FewBlocks b : {FewBlocks{1, 1}, FewBlocks{2, 1}, FewBlocks{4, 1}, FewBlocks{4, 2}})
    if ((b.nc == 1 || n.out_fp32 || n.K <= 2048) &&
        (b.channels(n) * b.tokens(n) <= 256 || (b.mt <= 2 && n.M <= 16 * b.mt)))
      return b;
  return {0, 0};
}

template <bool ROW, bool POW2, int OUT>
static void launch_linear_form(const Linear &n, const LinArgs &a, hipStream_t s) {
  const FewBlocks b = few_blocks(n);
  if (b.mt > 0) {
    const dim3 grid((unsigned)b.channels(n), (unsigned)b.tokens(n));
#define L(MT, NC) \
  hipLaunchKernelGGL((k_linear_fp8_few<MT, NC, ROW, POW2, OUT>), grid, dim3(64 * FewShape<MT>::waves), 0, s, a)
    if (b.mt == 1) L(1, 1);
    else if (b.mt == 2) L(2, 1);
    else if (b.nc == 1) L(4, 1);
    else L(4, 2);
#undef L
    return;
  }
  // the fastest tile by those times: of 333 x 4096 x 4096 64 x 64 (15.6 us; 128 x 128 24, 256 x 256
  // 42), of 512 x 7168 x 2048 128 x 128 (15; 64 x 64 18, 256 x 256 26), of 4096 x 4096 x 7168 256 x 256 (fp32
  // results: 128 x 192 where 1536 x 4096 x 16384 takes 173, 128 x 128 215)
  const bool fp32 = OUT == kOutFp32;
  using Large = std::conditional_t<OUT == kOutFp32, Shape128x192, Shape256>;
  const double large = tiles_time<Large>(n, fp32 ? TileTimes{1.3, 8.5, 0.0, 0.0} : TileTimes{1.6, 9.0, 0.0, 0.0}),
               mid = tiles_time<Shape128>(n, fp32 ? TileTimes{0.93, 7.0, 1.7, 6.0} : TileTimes{0.8, 1.5, 1.0, 6.0}),
               small = tiles_time<Shape64>(n, fp32 ? TileTimes{0.43, 4.0, 0.67, 4.0} : TileTimes{0.27, 3.0, 0.48, 3.0});
  if (large <= mid && large <= small) launch_tiles<Large, ROW, POW2, OUT>(a, fp32 ? 5 : 4, s);
  else if (mid <= small) launch_tiles<Shape128, ROW, POW2, OUT>(a, 8, s);
  else launch_tiles<Shape64, ROW, POW2, OUT>(a, 8, s);
}

// A launch counts its threads in 32 bits, and a tile index is an int32.
bool linear_fp8_fits(const Linear &n) {
  const FewBlocks b = few_blocks(n);
  if (b.mt > 0) return b.channels(n) * 512 < (int64_t)1 << 32 && b.tokens(n) <= 65535;
  return tiles_of(n, 64) + kXcds < (int64_t)1 << 24;
}

hipError_t launch_linear_fp8(const Linear &n, hipStream_t s) {
  if (n.M == 0 || n.N == 0) return hipSuccess;
  const LinArgs a{reinterpret_cast<const u32x4 *>(n.x), reinterpret_cast<const u32x4 *>(n.w), n.xs, n.ws,
                  n.addend, n.out, n.status, n.M, n.N, n.K};
#define L2(ROW, POW2)                                                   \
  do {                                                                  \
    if (n.glu) launch_linear_form<ROW, POW2, kOutGlu>(n, a, s);         \
    else if (n.out_fp32) launch_linear_form<ROW, POW2, kOutFp32>(n, a, s); \
    else launch_linear_form<ROW, POW2, kOutBf16>(n, a, s);              \
  } while (0)
  if (n.row_scales && n.pow2) L2(true, true);
  else if (n.row_scales) L2(true, false);
  else if (n.pow2) L2(false, true);
  else L2(false, false);
#undef L2
  return hipGetLastError();
}

}  // namespace epk
