// layernorm.hip -- residual addition, dropout of the branch and layer norm of
// token rows, with the rows handed on in bf16 and in 8 bits, and its backward,
// on gfx950.
//
//   h = round(dropout(x) + residual)      (the stream's type; x without both)
//   n = (h - mean) * rstd,  rstd = 1 / sqrt(mean((h - mean)^2) + eps)
//   y = n * w + b
//
// As in the RMS norm (norm.hip) the norm reads h as the stream stores it and
// the row is read once and stays in registers.  Mean and variance come from one
// reduction, of sum d and sum d^2 with d = h - c in fp64, c the row's first
// value: since c is one of the row's values, (mean - c)^2 is at most H times the
// variance, so the difference  sum d^2 - (sum d)^2 / H  loses at most a factor
// H of fp64's 2^-53, whatever the row's mean, and a constant row has variance 0
// exactly.  A second reduction, of the largest |y|, runs for INT8 rows only.
// Rows up to 2048 channels go one to a wave where there are many of them,
// others one to a workgroup.  Bound by memory where there are many rows (16384 x
// 4096 with dropout and a bf16 stream 99 us, 5.4 TB/s), by the latency of a load, a
// reduction and the stores where there are few (128 x 7168 to FP8 rows 5.1 us).
#include "ep_internal.h"
#include "philox.h"
#include "rows.h"

namespace epk {

// Sum of v over the workgroup (or the wave); two sums at once.
template <bool WAVE>
__device__ __forceinline__ void row_reduce2(double &u, double &v) {
  u = wave_sum(u);
  v = wave_sum(v);
  if constexpr (!WAVE) {
    __shared__ double s_sum[2][16];
    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6, nw = blockDim.x >> 6;
    if (lane == 0) {
      s_sum[0][wv] = u;
      s_sum[1][wv] = v;
    }
    __syncthreads();
    const int i = lane & 15;  // every 16-lane row reduces the waves' results
    u = row_sum(i < nw ? s_sum[0][i] : 0.0);
    v = row_sum(i < nw ? s_sum[1][i] : 0.0);
  }
}

// A sum of squares that rounding may have left below zero (a NaN stays one).
__device__ __forceinline__ double not_below_zero(double v) { return v < 0.0 ? 0.0 : v; }

template <typename T>
__device__ __forceinline__ float first_value(const void *p, int64_t v) {
  if constexpr (sizeof(T) == 2) return bf16_lo(static_cast<const uint16_t *>(p)[8 * v]);
  else return static_cast<const float *>(p)[8 * v];
}

// The branch's value joined with the stream: dropped ones leave the stream alone.
__device__ __forceinline__ float joined(float x, bool stay, float scale, float r) {
  return stay ? __builtin_fmaf(x, scale, r) : r;
}

template <typename RT>
__device__ __forceinline__ float as_stored(float h) {
  if constexpr (sizeof(RT) == 2) return bf16_lo(pack_bf16x2(h, 0.0f));
  else return h;
}

struct LnArgs {
  const u32x4 *x;
  const void *residual;  // bf16 or fp32 rows, or null
  const void *w, *b;     // b may be null
  void *hidden;          // or null
  u32x4 *y;              // or null
  u32x2 *codes;          // or null
  float *scales;
  int64_t T;             // rows
  int32_t V;             // vectors of 8 per row
  int32_t w_fp32, quant;
  double eps, inv_h;
  Dropout drop;
};

template <typename RT, bool RES, int VPT, bool WAVE>
__global__ __launch_bounds__(WAVE ? 256 : 1024) void k_add_layernorm(LnArgs a) {
  int sub, step;
  const int64_t row = my_row<WAVE>(sub, step), base = row * a.V;
  if (row >= a.T) return;  // the whole wave (and, with barriers, the workgroup)
  const bool drop = a.drop.rng != nullptr;
  const PhiloxKey key = drop ? philox_key(a.drop.rng) : PhiloxKey{};
  float h[VPT][8];
  u32x4 hb[VPT];  // bf16 rows: h as stored
  Raw8<uint16_t> xr[VPT];
  Raw8<RT> rr[VPT];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int32_t v = sub + i * step;
    if (v >= a.V) continue;
    xr[i] = load_raw<uint16_t, true>(a.x, base + v);
    if constexpr (RES) rr[i] = load_raw<RT, true>(a.residual, base + v);
  }
  // the row's first value, by every thread for itself
  const float x0 = first_value<uint16_t>(a.x, base), r0 = RES ? first_value<RT>(a.residual, base) : 0.0f;
  float c0 = RES ? x0 + r0 : x0;
  if (drop) c0 = joined(x0, stays(philox((uint64_t)base, key), 0, a.drop.threshold), a.drop.scale, r0);
  const double shift = (double)as_stored<RT>(c0);
  double s1 = 0.0, s2 = 0.0;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int32_t v = sub + i * step;
    if (v >= a.V) continue;
    unpack_raw(xr[i], h[i]);
    float r[8] = {};
    if constexpr (RES) unpack_raw(rr[i], r);
    if (drop) {
      const u32x4 bits = philox((uint64_t)(base + v), key);
#pragma unroll
      for (int c = 0; c < 8; ++c)
        h[i][c] = joined(h[i][c], stays(bits, c, a.drop.threshold), a.drop.scale, r[c]);
    } else if constexpr (RES) {
#pragma unroll
      for (int c = 0; c < 8; ++c) h[i][c] += r[c];
    }
    if constexpr (sizeof(RT) == 2) {   // as the stream will hold them
      hb[i] = pack8(h[i]);
      unpack8(hb[i], h[i]);
    }
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      const double d = (double)h[i][c] - shift;
      s1 += d;
      s2 = __builtin_fma(d, d, s2);
    }
  }
  row_reduce2<WAVE>(s1, s2);
  const double m1 = s1 * a.inv_h, mean = shift + m1;
  // half of h - mean, whose whole may lie outside fp32, times twice the reciprocal: the same roundings
  const double half_mean = 0.5 * mean;
  const float rstd2 = 2.0f * rstd_of(not_below_zero(__builtin_fma(-m1, s1, s2)), a.inv_h, a.eps);
  // the stream's rows are stored here, behind the reduction: they may replace
  // the residual, whose first value every thread reads.  Not read again before
  // the whole layer: past the caches, as the RMS norm's.
  if (a.hidden) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int32_t v = sub + i * step;
      if (v >= a.V) continue;
      if constexpr (sizeof(RT) == 2) {
        store_stream(static_cast<u32x4 *>(a.hidden) + base + v, hb[i]);
      } else {
        f32x4 *o = static_cast<f32x4 *>(a.hidden) + 2 * (base + v);
        store_stream(o, f32x4{h[i][0], h[i][1], h[i][2], h[i][3]});
        store_stream(o + 1, f32x4{h[i][4], h[i][5], h[i][6], h[i][7]});
      }
    }
  }
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int32_t v = sub + i * step;
    if (v >= a.V) continue;
    float w[8], b[8];
    load_weight8(a.w, a.w_fp32, v, w);
    if (a.b) load_weight8(a.b, a.w_fp32, v, b);
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      const float n = (float)__builtin_fma((double)h[i][c], 0.5, -half_mean) * rstd2;
      h[i][c] = a.b ? __builtin_fmaf(n, w[c], b[c]) : n * w[c];
      m = umax(m, magnitude_bits(h[i][c]));
    }
  }
  float s8 = 1.0f, inv8 = 1.0f;
  if (a.quant == kQuantInt8) {
    row_reduce<WAVE>(m);
    s8 = int8_scale(m);
    inv8 = 1.0f / s8;
    if (sub == 0) a.scales[row] = s8;
  }
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int32_t v = sub + i * step;
    if (v >= a.V) continue;
    if (a.y) a.y[base + v] = pack8(h[i]);
    if (a.quant == kQuantInt8) {
      a.codes[base + v] = m >= kInfBits ? u32x2{0u, 0u} : int8_codes(h[i], s8, inv8);
    } else if (a.quant != kQuantNone) {   // H % 128 == 0: a block's 16 lanes are all here
      float s;
      a.codes[base + v] = fp8_codes(h[i], &s, a.quant == kQuantFp8Pow2);
      if ((v & 15) == 0) a.scales[(base + v) >> 4] = s;
    }
  }
}

// As the RMS norm's, but rows of 4097 to 8192 channels count as many from two a compute unit on: its
// workgroups of 832 to 1024 threads fit once (4000 x 7168 31 us against 41, with bf16 stream and FP8
// rows 51 against 59; 1000 rows 10.0 against 12.3; 512 rows the same, 128 rows 5.7 against 5.1).
static RowShape ln_row_shape(int64_t rows, int32_t V) {
  return row_shape(V > 512 && V <= 1024 && rows > 512 ? INT32_MAX : rows, V);
}

hipError_t launch_add_layernorm(const LayerNorm &n, hipStream_t s) {
  if (n.T == 0) return hipSuccess;
  const LnArgs a{reinterpret_cast<const u32x4 *>(n.x), n.residual, n.w, n.b, n.hidden,
                 reinterpret_cast<u32x4 *>(n.y), reinterpret_cast<u32x2 *>(n.codes), n.scales,
                 n.T, n.H / 8, n.w_fp32 ? 1 : 0, n.quant, n.eps, 1.0 / n.H, n.drop};
  const RowShape sh = ln_row_shape(n.T, a.V);
#define L3(RT, RES, P, W) \
  hipLaunchKernelGGL((k_add_layernorm<RT, RES, P, W>), row_grid(n.T, W), dim3(sh.threads), 0, s, a)
#define LN(P, W) L3(uint16_t, false, P, W)
#define LB(P, W) L3(uint16_t, true, P, W)
#define LF(P, W) L3(float, true, P, W)
  if (!n.residual) EP_ROW_SWITCH(sh, LN);
  else if (n.res_fp32) EP_ROW_SWITCH(sh, LF);
  else EP_ROW_SWITCH(sh, LB);
#undef LF
#undef LB
#undef LN
#undef L3
  return hipGetLastError();
}

// ---------------------------------------------------------------------------
// backward
//
// With n as above and g = grad_y * w:
//   grad_h = rstd * (g - mean(g) - n * mean(g * n)) [+ grad_hidden]
//   grad_x = dropout(grad_h)
//   grad_w = sum over rows of grad_y * n,  grad_b = sum over rows of grad_y
// One reduction over a row gives its four sums, d = h - c as in the forward:
// sum d, sum d^2, sum g and sum g * d; sum g * n follows from the last two.  g is
// exact in fp64: means of terms that cancel keep no rounding of theirs.
// A workgroup takes every G-th row (or group of rows), the next row's loads in
// flight while one is reduced, and keeps its share of grad_w and grad_b in
// registers, in fp32: T / 512 rows, T / 256 above 4096 channels, so that 16384 rows
// are 32 or 64 additions of half a step each at most.  The G partial rows, both side
// by side, go to the workspace and norm.hip's second kernel adds them in order, in
// fp64.  They are twice as long as the RMS norm's, so there are no more workgroups of
// over 512 threads than compute units (one fits: 4096 x 7168 with dropout 74 us
// against 79 with up to 512), and fp32 rows of 2049 to 4096 channels go two to a
// workgroup of up to 1024 threads (16384 x 4096 200 us against 210; bf16 rows 152
// against 147, one to a workgroup).

static BwdShape ln_bwd_shape(int32_t V, bool fp32) {
  BwdShape b = bwd_shape(V);
  if (fp32 && b.threads > 256 && b.threads <= 512) b.rows = 2;
  return b;
}

static int32_t ln_bwd_groups(int32_t T, int32_t V, bool fp32) {
  if (T == 0) return 0;
  const BwdShape b = ln_bwd_shape(V, fp32);
  const int64_t units = ((int64_t)T + b.rows - 1) / b.rows, most = b.threads * b.rows > 512 ? 256 : 512;
  int64_t passes = (units + most - 1) / most;
  if (passes < 2 && units > 256) passes = 2;
  return (int32_t)((units + passes - 1) / passes);
}

int32_t layernorm_bwd_groups(int32_t T, int32_t H) {
  const int32_t a = ln_bwd_groups(T, H / 8, false), b = ln_bwd_groups(T, H / 8, true);
  return a > b ? a : b;
}

struct LnBwdArgs {
  const void *hidden;
  const void *w;
  const u32x4 *gy;
  const void *ghidden;  // or null
  void *gh;             // or null (grad_x alone)
  u32x4 *gx;            // or null
  float *part;          // [G][2 H] partial grad_w and grad_b, or null
  int32_t T, V, w_fp32, rows;
  double eps, inv_h;
  Dropout drop;
};

template <typename RT, int VPT>
__global__ __launch_bounds__(1024) void k_layernorm_bwd(LnBwdArgs a) {
  __shared__ double s_sum[2][4][16];
  extern __shared__ float s_dw[];  // [rows - 1][2 H]
  // (a wave's threads are of one row: said so, the row and its offsets take no vector registers)
  const int tpr = blockDim.x / a.rows, slot = __builtin_amdgcn_readfirstlane(threadIdx.x / tpr);
  const int sub = threadIdx.x - slot * tpr;
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6, nw = tpr >> 6, w0 = slot * nw;
  const bool drop = a.gx != nullptr;
  const PhiloxKey key = drop ? philox_key(a.drop.rng) : PhiloxKey{};
  // one vector a thread: the next row's loads in flight under this row, and the weight in registers.
  // More: the row is read again behind the reduction, out of the L2, for registers that spill cost more
  // (held packed, 4096 x 12288 with dropout takes 154 us in bf16 and 207 in fp32 against 131 and 195).
  // Above 16384 channels the two sums alone are 64 registers: 64 (bf16) and 63 (fp32) of all spill, and
  // 2048 x 20480 takes 202 and 227 us, 40 and 57% of the copy rate
  constexpr bool AHEAD = VPT == 1;
  float w[8], dw[VPT][8], db[VPT][8];
  Raw8<RT> hr, rr;
  u32x4 gr;
  float first = 0.0f;
  const auto load = [&](int64_t t) {
    if (t >= a.T) return;
    const int64_t base = t * a.V;
    first = first_value<RT>(a.hidden, base);
    if (!AHEAD || sub >= a.V) return;
    hr = load_raw<RT, true>(a.hidden, base + sub);
    gr = load_stream(a.gy + base + sub);
    if (a.ghidden) rr = load_raw<RT, true>(a.ghidden, base + sub);
  };
  const int64_t step = (int64_t)gridDim.x * a.rows;
  int64_t t = (int64_t)blockIdx.x * a.rows + slot;
  if constexpr (AHEAD) {
    load(t);
    if (sub < a.V) load_weight8(a.w, a.w_fp32, sub, w);
  }
#pragma unroll
  for (int i = 0; i < VPT; ++i)
#pragma unroll
    for (int c = 0; c < 8; ++c) dw[i][c] = db[i][c] = 0.0f;
  int buf = 0;
  // (all rows of the workgroup go through the same passes: the barrier)
  for (; t - slot < a.T; t += step, buf ^= 1) {
    const int64_t base = t * a.V;
    const bool live = t < a.T;
    float h[8] = {}, g[8] = {}, r[8] = {};
    double s[4] = {0.0, 0.0, 0.0, 0.0};
    if constexpr (!AHEAD) load(t);
    const double shift = (double)first;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int32_t v = sub + i * tpr;
      if (v >= a.V || !live) continue;
      if constexpr (AHEAD) {
        unpack_raw(hr, h);
        unpack8(gr, g);
        if (a.ghidden) unpack_raw(rr, r);
      } else {
        unpack_raw(load_raw<RT, false>(a.hidden, base + v), h);
        unpack8(a.gy[base + v], g);
        load_weight8(a.w, a.w_fp32, v, w);
      }
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        const double d = (double)h[c] - shift, gw = (double)g[c] * (double)w[c];
        s[0] += d;
        s[1] = __builtin_fma(d, d, s[1]);
        s[2] += gw;
        s[3] = __builtin_fma(gw, d, s[3]);
      }
    }
    if constexpr (AHEAD) load(t + step);
#pragma unroll
    for (int q = 0; q < 4; ++q) s[q] = wave_sum(s[q]);
    if (nw > 1) {
      if (lane == 0) {
#pragma unroll
        for (int q = 0; q < 4; ++q) s_sum[buf][q][wv] = s[q];
      }
      __syncthreads();   // two buffers: the next row's sums do not meet this row's readers
      const int i = lane & 15;
#pragma unroll
      for (int q = 0; q < 4; ++q) s[q] = row_sum(i < nw ? s_sum[buf][q][w0 + i] : 0.0);
    }
    const double m1 = s[0] * a.inv_h, mean = shift + m1;
    const float rstd = rstd_of(not_below_zero(__builtin_fma(-m1, s[0], s[1])), a.inv_h, a.eps);
    // n = (h - mean) * rstd with the mean in two floats: no step of n is wider than fp32 (nor larger: half
    // of h - mean times twice rstd, as in the forward)
    const float mh = (float)mean, ml = (float)(mean - (double)mh) * rstd, mh2 = 0.5f * mh, rstd2 = 2.0f * rstd;
    const float mg = (float)(s[2] * a.inv_h);
    const float mn = (float)(__builtin_fma(-m1, s[2], s[3]) * (double)rstd * a.inv_h);  // mean of g * n
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int32_t v = sub + i * tpr;
      if (v >= a.V || !live) continue;
      if constexpr (!AHEAD) {
        unpack_raw(load_raw<RT, true>(a.hidden, base + v), h);
        unpack8(load_stream(a.gy + base + v), g);
        load_weight8(a.w, a.w_fp32, v, w);
        if (a.ghidden) unpack_raw(load_raw<RT, true>(a.ghidden, base + v), r);
      }
      float o[8];
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        const float n = __builtin_fmaf(__builtin_fmaf(h[c], 0.5f, -mh2), rstd2, -ml);
        o[c] = rstd * ((g[c] * w[c] - mg) - n * mn) + r[c];
        dw[i][c] += g[c] * n;
        db[i][c] += g[c];
      }
      if (a.gh) store8<RT>(a.gh, base + v, o);
      if (drop) {
        const u32x4 bits = philox((uint64_t)(base + v), key);
#pragma unroll
        for (int c = 0; c < 8; ++c) o[c] = stays(bits, c, a.drop.threshold) ? o[c] * a.drop.scale : 0.0f;
        a.gx[base + v] = pack8(o);
      }
    }
  }
  if (!a.part) return;
  if constexpr (VPT == 1) {   // several rows only with one vector a thread; joined in fp64
    if (a.rows > 1) {
      const int32_t H = a.V * 8;
      if (slot > 0 && sub < a.V) {
        float *o = s_dw + (slot - 1) * 2 * H;
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          o[c * a.V + sub] = dw[0][c];
          o[H + c * a.V + sub] = db[0][c];
        }
      }
      __syncthreads();
      if (slot > 0) return;
      if (sub < a.V) {
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          double sw = (double)dw[0][c], sb = (double)db[0][c];
          for (int i = 0; i < a.rows - 1; ++i) {
            sw += (double)s_dw[i * 2 * H + c * a.V + sub];
            sb += (double)s_dw[i * 2 * H + H + c * a.V + sub];
          }
          dw[0][c] = (float)sw;
          db[0][c] = (float)sb;
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int32_t v = sub + i * tpr;
    if (v >= a.V) continue;
    store8<float>(a.part, (int64_t)blockIdx.x * 2 * a.V + v, dw[i]);
    store8<float>(a.part, (int64_t)blockIdx.x * 2 * a.V + a.V + v, db[i]);
  }
}

hipError_t launch_layernorm_bwd(const LayerNormBwd &n, hipStream_t s) {
  const int32_t G = ln_bwd_groups(n.T, n.H / 8, n.h_fp32);
  if (n.T > 0) {
    const BwdShape sh = ln_bwd_shape(n.H / 8, n.h_fp32);
    const bool sums = n.gw || n.gb;
    const LnBwdArgs a{n.hidden, n.w, reinterpret_cast<const u32x4 *>(n.gy), n.ghidden, n.gh,
                      reinterpret_cast<u32x4 *>(n.gx), sums ? n.part : nullptr, n.T, n.H / 8,
                      n.w_fp32 ? 1 : 0, sh.rows, n.eps, 1.0 / n.H, n.drop};
    const size_t lds = sizeof(float) * 2 * (size_t)(sh.rows - 1) * n.H;   // 32 KB at most
#define L2(RT, P)                                                                               \
  hipLaunchKernelGGL((k_layernorm_bwd<RT, P>), dim3((unsigned)G), dim3(sh.threads * sh.rows), lds, \
                     s, a)
#define L(RT)                       \
  do {                              \
    if (sh.vpt == 1) L2(RT, 1);     \
    else if (sh.vpt == 2) L2(RT, 2); \
    else L2(RT, 4);                 \
  } while (0)
    if (n.h_fp32) L(float);
    else L(uint16_t);
#undef L
#undef L2
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (!n.gw && !n.gb) return hipSuccess;
  return launch_norm_dw(n.part, G, 2 * n.H, n.H, n.gw, n.gb, s);   // T == 0: zeros
}

}  // namespace epk
