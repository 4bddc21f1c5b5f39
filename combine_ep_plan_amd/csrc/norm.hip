// norm.hip -- the residual addition and RMS norm before an MoE layer, with the
// rows it hands on in bf16 and in 8 bits, its backward, and the INT8 row
// quantiser, on gfx950.
//
//   h = round(x + residual)       (the stream's type; h = x without a residual)
//   y = (h * w) * rstd,  rstd = 1 / sqrt(mean(h^2) + eps)
//
// The norm reads h as the stream stores it, so that the backward and the next
// layer, which read the stored stream, see the very rows that were
// normalised.  The sum of squares runs in fp64 and rstd is rounded once to
// fp32: its value does not depend on the order of the sum, so the 8-bit codes,
// which are decided in fp32, are the same on any implementation of these
// formulas.  The largest |y| is (largest |h * w|) * rstd, so one reduction
// over the row gives both rstd and the INT8 scale, and the row is read once and
// stays in registers.
//
// Rows: up to 2048 channels go one to a wave (four to a workgroup, no barrier);
// longer ones one to a workgroup.
#include "ep_internal.h"
#include "int8.h"
#include "lanes.h"

namespace epk {

enum Quant : int32_t { kQuantNone = 0, kQuantFp8 = 1, kQuantFp8Pow2 = 2, kQuantInt8 = 3 };

struct NormArgs {
  const u32x4 *x;
  const void *residual;  // bf16 or fp32 rows, or null
  const void *w;
  void *hidden;
  u32x4 *y;        // or null
  u32x2 *codes;    // or null
  float *scales;
  int64_t T;       // rows
  int32_t V;       // vectors of 8 per row
  int32_t w_fp32, quant;
  double eps, inv_h;
};

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

// FP8 codes of eight values of y whose 128-channel block spans 16 lanes; the
// FP8 dispatch's recipe (quantize_fp8_vec in dispatch.hip) on fp32 values.  The
// correctly rounded quotient y / s without a division each: with inv = 1 / s
// correctly rounded, q = y * inv corrected once by its exact remainder is
// y / s rounded (Markstein, "Computation of elementary functions on the IBM
// RISC System/6000 processor", 1990), where nothing underflows: blocks of tiny
// values divide.
__device__ __forceinline__ u32x2 fp8_codes(const float y[8], float *scale, bool pow2) {
  uint32_t a = 0;
#pragma unroll
  for (int c = 0; c < 8; ++c) a = umax(a, magnitude_bits(y[c]));
  a = row_max(a);
  float s = fp8_scale(a);
  if (pow2 && a != 0u && a < kInfBits) {
    const uint32_t b = __float_as_uint(s);   // subnormal ones end at 2^-126
    if (b & 0x007FFFFFu) s = __uint_as_float((b & 0x7F800000u) + 0x00800000u);
  }
  *scale = s;
  if (a >= kInfBits) return u32x2{0u, 0u};
  float q[8];
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
  uint32_t w0 = __builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], 0, false);
  w0 = __builtin_amdgcn_cvt_pk_fp8_f32(q[2], q[3], w0, true);
  uint32_t w1 = __builtin_amdgcn_cvt_pk_fp8_f32(q[4], q[5], 0, false);
  w1 = __builtin_amdgcn_cvt_pk_fp8_f32(q[6], q[7], w1, true);
  return u32x2{w0, w1};
}

// Workgroups of a launch over rows, RPB rows each: a launch counts its threads
// in 32 bits, so many rows spread over the grid's second dimension too.
constexpr int kRowWaves4 = 4;  // rows of a workgroup with a wave to a row
static dim3 row_grid(int64_t rows, bool wave) {
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

template <typename RT, bool RES, int VPT, bool WAVE>
__global__ __launch_bounds__(WAVE ? 256 : 1024) void k_add_rmsnorm(NormArgs a) {
  int sub, step;
  const int64_t row = my_row<WAVE>(sub, step), base = row * a.V;
  if (row >= a.T) return;  // the whole wave (and, with barriers, the workgroup)
  float p[VPT][8];  // h, then h * w
  Raw8<uint16_t> xr[VPT];
  Raw8<RT> rr[VPT];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int32_t v = sub + i * step;
    if (v >= a.V) continue;
    xr[i] = load_raw<uint16_t, true>(a.x, base + v);
    if constexpr (RES) rr[i] = load_raw<RT, true>(a.residual, base + v);
  }
  double ss = 0.0;
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int32_t v = sub + i * step;
    if (v >= a.V) continue;
    float h[8], w[8];
    unpack_raw(xr[i], h);
    load_weight8(a.w, a.w_fp32, v, w);
    if constexpr (RES) {
      float r[8];
      unpack_raw(rr[i], r);
#pragma unroll
      for (int c = 0; c < 8; ++c) h[c] += r[c];
      // the stream is next read behind the whole MoE layer: its rows leave no
      // lines behind (prefill 4096 x 7168, FP8: 49.5 us against 54)
      if constexpr (sizeof(RT) == 2) {
        const u32x4 b = pack8(h);
        store_stream(static_cast<u32x4 *>(a.hidden) + base + v, b);
        unpack8(b, h);
      } else {
        f32x4 *o = static_cast<f32x4 *>(a.hidden) + 2 * (base + v);
        store_stream(o, f32x4{h[0], h[1], h[2], h[3]});
        store_stream(o + 1, f32x4{h[4], h[5], h[6], h[7]});
      }
    }
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      ss = __builtin_fma((double)h[c], (double)h[c], ss);
      p[i][c] = h[c] * w[c];
      m = umax(m, magnitude_bits(p[i][c]));
    }
  }
  row_reduce<WAVE>(ss, m);
  const float rstd = rstd_of(ss, a.inv_h, a.eps);
  const uint32_t am = magnitude_bits(__uint_as_float(m) * rstd);
  const float s8 = int8_scale(am), inv8 = 1.0f / s8;
  if (a.quant == kQuantInt8 && sub == 0) a.scales[row] = s8;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int32_t v = sub + i * step;
    if (v >= a.V) continue;
    float y[8];
#pragma unroll
    for (int c = 0; c < 8; ++c) y[c] = p[i][c] * rstd;
    if (a.y) a.y[base + v] = pack8(y);
    if (a.quant == kQuantInt8) {
      a.codes[base + v] = am >= kInfBits ? u32x2{0u, 0u} : int8_codes(y, s8, inv8);
    } else if (a.quant != kQuantNone) {   // H % 128 == 0: a block's 16 lanes are all here
      float s;
      a.codes[base + v] = fp8_codes(y, &s, a.quant == kQuantFp8Pow2);
      if ((v & 15) == 0) a.scales[(base + v) >> 4] = s;
    }
  }
}

// Threads of a row of V vectors (V <= 4096) and vectors a thread.
struct RowShape {
  bool wave;
  int threads, vpt;
};
// Few rows (latency counts) get a thread to a vector where 1024 threads allow
// it: INT8 rows of 1024 x 2048 4.1 us against 5.0 with a wave to a row.  Many
// rows: a wave each up to 2048 channels, 33 us against 47 with a workgroup each
// for 32768 x 2048 (no barrier, more loads in flight).
constexpr int64_t kFewRows = 4096;
static RowShape row_shape(int64_t rows, int32_t V) {
  if (rows < kFewRows && V <= 1024) return {false, (V + 63) / 64 * 64, 1};
  if (V <= 256) return {true, 256, V <= 64 ? 1 : V <= 128 ? 2 : 4};
  const int threads = V <= 512 ? 256 : V <= 1024 ? 512 : 1024;
  return {false, threads, V <= 2 * threads ? 2 : 4};
}
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

hipError_t launch_add_rmsnorm(const RmsNorm &n, hipStream_t s) {
  if (n.T == 0) return hipSuccess;
  const NormArgs a{reinterpret_cast<const u32x4 *>(n.x), n.residual, n.w, n.hidden,
                   reinterpret_cast<u32x4 *>(n.y), reinterpret_cast<u32x2 *>(n.codes), n.scales,
                   n.T, n.H / 8, n.w_fp32 ? 1 : 0, n.quant, n.eps, 1.0 / n.H};
  const RowShape sh = row_shape(n.T, a.V);
#define L3(RT, RES, P, W) \
  hipLaunchKernelGGL((k_add_rmsnorm<RT, RES, P, W>), row_grid(n.T, W), dim3(sh.threads), 0, s, a)
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
// With n = h * rstd and g = grad_y * w:
//   grad_h = rstd * (g - n * mean(g * n)) [+ grad_hidden]
//   grad_w = sum over rows of grad_y * n
// One reduction over a row gives sum h^2 and sum g * h.  A workgroup takes
// every G-th row (or group of narrow rows), the next row's loads in flight while
// one is reduced, and keeps its share of grad_w in registers; the G partial rows
// go to the workspace and a second kernel adds them in order, in fp64, so the
// result does not depend on scheduling.  16384 x 4096: 90 + 5 us, 5.9 TB/s.

// Threads of a backward row, vectors a thread, rows a workgroup takes at a time
// (narrow rows share one, so that there are few partial rows of grad_w).  Rows
// longer than 8192 channels have two or four vectors a thread and 1024 threads,
// whose 128 registers do not hold them: 22 and 183 are spilled in bf16, 38 and 318
// in fp32 (4096 x 12288: 132 and 243 us, 3.0 TB/s; 4096 x 20480: 610 and 811).
struct BwdShape {
  int threads, vpt, rows;
};
static BwdShape bwd_shape(int32_t V) {
  BwdShape b;
  b.threads = V <= 1024 ? (V + 63) / 64 * 64 : 1024;
  b.vpt = V <= b.threads ? 1 : V <= 2 * b.threads ? 2 : 4;
  b.rows = b.threads <= 256 ? 512 / b.threads : 1;
  return b;
}

// Workgroups of the backward: up to 512 (two of 512 threads a compute unit),
// each with as many passes as the others, and at least two where there are rows
// enough for 256 of them: a partial row costs as much to write and read as half
// a row of the inputs.
int32_t norm_bwd_groups(int32_t T, int32_t H) {
  if (T == 0) return 0;
  const int64_t units = ((int64_t)T + bwd_shape(H / 8).rows - 1) / bwd_shape(H / 8).rows;
  int64_t passes = (units + 511) / 512;
  if (passes < 2 && units > 256) passes = 2;
  return (int32_t)((units + passes - 1) / passes);
}

struct NormBwdArgs {
  const void *hidden;
  const void *w;
  const u32x4 *gy;
  const void *ghidden;  // or null
  void *gx;
  float *part;          // [G][H] partial grad_w, or null
  int32_t T, V, w_fp32, rows;
  double eps, inv_h;
};

template <typename RT, int VPT>
__global__ __launch_bounds__(1024) void k_rmsnorm_bwd(NormBwdArgs a) {
  __shared__ double s_sum[2][2][16];
  extern __shared__ double s_dw[];  // [rows - 1][H]
  const int tpr = blockDim.x / a.rows, slot = threadIdx.x / tpr, sub = threadIdx.x - slot * tpr;
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6, nw = tpr >> 6, w0 = slot * nw;
  // the next row's loads in flight under this row, and the weight in registers,
  // where they fit
  constexpr bool AHEAD = VPT == 1;
  float w[VPT][8], dw[VPT][8];
  Raw8<RT> hr[VPT], rr[VPT];
  u32x4 gr[VPT];
  const auto load = [&](int64_t t) {
    const int64_t base = t * a.V;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int32_t v = sub + i * tpr;
      if (v >= a.V || t >= a.T) continue;
      hr[i] = load_raw<RT, true>(a.hidden, base + v);
      gr[i] = load_stream(a.gy + base + v);
      if (a.ghidden) rr[i] = load_raw<RT, true>(a.ghidden, base + v);
    }
  };
  const auto weight = [&] {
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int32_t v = sub + i * tpr;
      if (v < a.V) load_weight8(a.w, a.w_fp32, v, w[i]);
    }
  };
  const int64_t step = (int64_t)gridDim.x * a.rows;
  int64_t t = (int64_t)blockIdx.x * a.rows + slot;
  if constexpr (AHEAD) {
    load(t);
    weight();
  }
#pragma unroll
  for (int i = 0; i < VPT; ++i)
#pragma unroll
    for (int c = 0; c < 8; ++c) dw[i][c] = 0.0f;
  int buf = 0;
  // (all rows of the workgroup go through the same passes: the barrier)
  for (; t - slot < a.T; t += step, buf ^= 1) {
    const int64_t base = t * a.V;
    const bool live = t < a.T;
    float h[VPT][8], g[VPT][8], r[VPT][8];
    double ss = 0.0, sg = 0.0;
    if constexpr (!AHEAD) {
      load(t);
      weight();
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int32_t v = sub + i * tpr;
#pragma unroll
      for (int c = 0; c < 8; ++c) h[i][c] = g[i][c] = r[i][c] = 0.0f;
      if (v >= a.V || !live) continue;
      unpack_raw(hr[i], h[i]);
      unpack8(gr[i], g[i]);
      if (a.ghidden) unpack_raw(rr[i], r[i]);
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        ss = __builtin_fma((double)h[i][c], (double)h[i][c], ss);
        sg = __builtin_fma((double)(g[i][c] * w[i][c]), (double)h[i][c], sg);
      }
    }
    if constexpr (AHEAD) load(t + step);
    ss = wave_sum(ss);
    sg = wave_sum(sg);
    if (nw > 1) {
      if (lane == 0) {
        s_sum[buf][0][wv] = ss;
        s_sum[buf][1][wv] = sg;
      }
      __syncthreads();   // two buffers: the next row's sums do not meet this row's readers
      const int i = lane & 15;
      ss = row_sum(i < nw ? s_sum[buf][0][w0 + i] : 0.0);
      sg = row_sum(i < nw ? s_sum[buf][1][w0 + i] : 0.0);
    }
    const float rstd = rstd_of(ss, a.inv_h, a.eps);
    const float mean = (float)(sg * (double)rstd * a.inv_h);  // mean of g * n
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int32_t v = sub + i * tpr;
      if (v >= a.V || !live) continue;
      float o[8];
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        const float n = h[i][c] * rstd;
        o[c] = rstd * (g[i][c] * w[i][c] - n * mean) + r[i][c];
        dw[i][c] += g[i][c] * n;
      }
      // cached: the next backward reads it (a chain of these calls on 16384 x
      // 4096 takes 85 us a call, 95 with streaming stores)
      store8<RT>(a.gx, base + v, o);
    }
  }
  if (!a.part) return;
  if constexpr (VPT == 1) {   // several rows only with one vector a thread; joined in fp64
    if (a.rows > 1) {
      const int32_t H = a.V * 8;
      if (slot > 0 && sub < a.V) {
#pragma unroll
        for (int c = 0; c < 8; ++c) s_dw[(slot - 1) * H + c * a.V + sub] = (double)dw[0][c];
      }
      __syncthreads();
      if (slot > 0) return;
      if (sub < a.V) {
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          double sum = (double)dw[0][c];
          for (int i = 0; i < a.rows - 1; ++i) sum += s_dw[i * H + c * a.V + sub];
          dw[0][c] = (float)sum;
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int32_t v = sub + i * tpr;
    if (v < a.V) store8<float>(a.part, (int64_t)blockIdx.x * a.V + v, dw[i]);
  }
}

// grad_w[c] = sum of the G partial rows: a workgroup takes 32 columns, its 32
// thread rows every 32nd partial row each, all fp64, joined
// in order.
constexpr int kDwThreads = 1024, kDwCols = 32, kDwRows = kDwThreads / kDwCols;
__global__ __launch_bounds__(kDwThreads) void k_rmsnorm_dw(const float *__restrict__ part, int32_t G,
                                                           int32_t H, float *__restrict__ dw) {
  __shared__ double s[kDwRows][kDwCols];
  const int cl = threadIdx.x % kDwCols, rl = threadIdx.x / kDwCols;
  const int32_t c = blockIdx.x * kDwCols + cl;
  double sum = 0.0;
  if (c < H) {
    int32_t i = rl;
    for (; i + 7 * kDwRows < G; i += 8 * kDwRows) {
      float v[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) v[u] = part[(int64_t)(i + u * kDwRows) * H + c];
#pragma unroll
      for (int u = 0; u < 8; ++u) sum += (double)v[u];
    }
    for (; i < G; i += kDwRows) sum += (double)part[(int64_t)i * H + c];
  }
  s[rl][cl] = sum;
  __syncthreads();
  // halves: thread row r adds row r + n's sum, for n = kDwRows / 2, ..., 1
  for (int n = kDwRows / 2; n > 0; n >>= 1) {
    if (rl < n) s[rl][cl] += s[rl + n][cl];
    __syncthreads();
  }
  if (rl == 0 && c < H) dw[c] = (float)s[0][cl];
}

hipError_t launch_rmsnorm_bwd(const RmsNormBwd &n, hipStream_t s) {
  const int32_t G = norm_bwd_groups(n.T, n.H);
  if (n.T > 0) {
    const BwdShape sh = bwd_shape(n.H / 8);
    const NormBwdArgs a{n.hidden, n.w, reinterpret_cast<const u32x4 *>(n.gy), n.ghidden, n.gx,
                        n.gw ? n.part : nullptr, n.T, n.H / 8, n.w_fp32 ? 1 : 0, sh.rows, n.eps,
                        1.0 / n.H};
    const size_t lds = sizeof(double) * (size_t)(sh.rows - 1) * n.H;   // 28 KB at most
#define L2(RT, P)                                                                             \
  hipLaunchKernelGGL((k_rmsnorm_bwd<RT, P>), dim3((unsigned)G), dim3(sh.threads * sh.rows), lds, \
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
  if (!n.gw) return hipSuccess;
  hipLaunchKernelGGL(k_rmsnorm_dw, dim3((unsigned)((n.H + kDwCols - 1) / kDwCols)), dim3(kDwThreads),
                     0, s, n.part, G, n.H, n.gw);   // T == 0: zeros
  return hipGetLastError();
}

// ---------------------------------------------------------------------------
// INT8 rows from bf16 rows (the activation between an expert FFN's two INT8
// products): the row in registers between the reduction of its amax and its
// codes.

template <int VPT, bool WAVE>
__global__ __launch_bounds__(WAVE ? 256 : 1024) void k_quantize_int8(const u32x4 *__restrict__ x,
                                                                     u32x2 *__restrict__ codes,
                                                                     float *__restrict__ scales,
                                                                     int64_t rows, int32_t V) {
  int sub, step;
  const int64_t row = my_row<WAVE>(sub, step), base = row * V;
  if (row >= rows) return;
  u32x4 r[VPT];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int32_t v = sub + i * step;
    r[i] = v < V ? load_stream(x + base + v) : u32x4{0u, 0u, 0u, 0u};
  }
  // bf16 magnitudes order like their bits: two at a time in the halves of a word
  uint32_t hi = 0, lo = 0;
#pragma unroll
  for (int i = 0; i < VPT; ++i)
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const uint32_t b = r[i][c] & 0x7FFF7FFFu;
      hi = umax(hi, b);
      lo = umax(lo, b << 16);
    }
  uint32_t m = umax(hi & 0xFFFF0000u, lo);
  row_reduce<WAVE>(m);
  const float s = int8_scale(m), inv = 1.0f / s;
  if (sub == 0) scales[row] = s;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int32_t v = sub + i * step;
    if (v >= V) continue;
    float f[8];
    unpack8(r[i], f);
    codes[base + v] = m >= kInfBits ? u32x2{0u, 0u} : int8_codes(f, s, inv);
  }
}

hipError_t launch_quantize_int8(const uint16_t *x, int64_t rows, int32_t K, uint8_t *codes,
                                float *scales, hipStream_t s) {
  if (rows == 0) return hipSuccess;
  const int32_t V = K / 8;
  const RowShape sh = row_shape(rows, V);
#define L(P, W)                                                                            \
  hipLaunchKernelGGL((k_quantize_int8<P, W>), row_grid(rows, W), dim3(sh.threads), 0, s,   \
                     reinterpret_cast<const u32x4 *>(x), reinterpret_cast<u32x2 *>(codes), \
                     scales, rows, V)
  EP_ROW_SWITCH(sh, L);
#undef L
  return hipGetLastError();
}

}  // namespace epk
