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
#include "ep_internal.h"
#include "int8.h"

namespace epk {

constexpr int kNormMaxVec = 4;  // 16-byte vectors of bf16 a thread holds
enum Quant : int32_t { kQuantNone = 0, kQuantFp8 = 1, kQuantFp8Pow2 = 2, kQuantInt8 = 3 };

struct NormArgs {
  const u32x4 *x;
  const void *residual;  // bf16 or fp32 rows, or null
  const void *w;
  void *hidden;
  u32x4 *y;        // or null
  u32x2 *codes;    // or null
  float *scales;
  int32_t T, V;    // rows, vectors of 8 per row
  int32_t w_fp32, quant;
  double eps;
};

// Eight values of a bf16 or fp32 row.
template <typename T>
__device__ __forceinline__ void load8(const void *p, int64_t v, float f[8]) {
  if constexpr (sizeof(T) == 2) {
    unpack8(static_cast<const u32x4 *>(p)[v], f);
  } else {
    const f32x4 a = static_cast<const f32x4 *>(p)[2 * v], b = static_cast<const f32x4 *>(p)[2 * v + 1];
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
  }
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

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d);
  return v;
}

__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) {
    const uint32_t o = (uint32_t)__shfl_xor((int)v, d);
    v = o > v ? o : v;
  }
  return v;
}

// rstd of a row from its sum of squares.
__device__ __forceinline__ float rstd_of(double ss, int32_t H, double eps) {
  return (float)(1.0 / sqrt(ss / (double)H + eps));
}

// FP8 codes of eight values of y whose 128-channel block spans 16 lanes; the
// FP8 dispatch's recipe (quantize_fp8_vec in dispatch.hip) on fp32 values.
__device__ __forceinline__ u32x2 fp8_codes(const float y[8], float *scale, bool pow2) {
  uint32_t a = 0;
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    const uint32_t m = magnitude_bits(y[c]);
    a = m > a ? m : a;
  }
#pragma unroll
  for (int d = 8; d > 0; d >>= 1) {
    const uint32_t o = (uint32_t)__shfl_xor((int)a, d);
    a = o > a ? o : a;
  }
  float s = fp8_scale(a);
  if (pow2 && a != 0u && a < kInfBits) {
    const uint32_t b = __float_as_uint(s);
    if (b & 0x007FFFFFu) s = __uint_as_float((b & 0x7F800000u) + 0x00800000u);
  }
  *scale = s;
  if (a >= kInfBits) return u32x2{0u, 0u};
  float q[8];
#pragma unroll
  for (int c = 0; c < 8; ++c) q[c] = fminf(fmaxf(y[c] / s, -448.0f), 448.0f);
  uint32_t w0 = __builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], 0, false);
  w0 = __builtin_amdgcn_cvt_pk_fp8_f32(q[2], q[3], w0, true);
  uint32_t w1 = __builtin_amdgcn_cvt_pk_fp8_f32(q[4], q[5], 0, false);
  w1 = __builtin_amdgcn_cvt_pk_fp8_f32(q[6], q[7], w1, true);
  return u32x2{w0, w1};
}

// Row of a workgroup: a launch counts its threads in 32 bits, so many rows
// spread over the grid's second dimension too.
constexpr int64_t kGridRows = 1 << 20;
__device__ __forceinline__ int64_t grid_row() { return (int64_t)blockIdx.y * gridDim.x + blockIdx.x; }
static dim3 row_grid(int64_t rows) {
  const int64_t gx = rows < kGridRows ? rows : kGridRows;
  return dim3((unsigned)gx, (unsigned)((rows + gx - 1) / gx));
}

// One workgroup per row; a thread holds VPT vectors of it.
template <typename RT, bool RES, int VPT>
__global__ __launch_bounds__(1024) void k_add_rmsnorm(NormArgs a) {
  __shared__ double s_sum[16];
  __shared__ uint32_t s_max[16];
  const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6, nw = blockDim.x >> 6;
  const int64_t row = grid_row(), base = row * a.V;
  if (row >= a.T) return;
  float p[VPT][8];  // h * w
  double ss = 0.0;
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int32_t v = tid + i * blockDim.x;
    if (v >= a.V) continue;
    float h[8], w[8];
    load8<uint16_t>(a.x, base + v, h);
    if constexpr (RES) {
      float r[8];
      load8<RT>(a.residual, base + v, r);
#pragma unroll
      for (int c = 0; c < 8; ++c) h[c] += r[c];
      if constexpr (sizeof(RT) == 2) {
        const u32x4 b = pack8(h);
        static_cast<u32x4 *>(a.hidden)[base + v] = b;
        unpack8(b, h);
      } else {
        store8<RT>(a.hidden, base + v, h);
      }
    }
    load_weight8(a.w, a.w_fp32, v, w);
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      ss += (double)h[c] * (double)h[c];
      p[i][c] = h[c] * w[c];
      const uint32_t b = magnitude_bits(p[i][c]);
      m = b > m ? b : m;
    }
  }
  ss = wave_sum(ss);
  m = wave_max(m);
  if (lane == 0) {
    s_sum[wv] = ss;
    s_max[wv] = m;
  }
  __syncthreads();
  ss = 0.0;
  m = 0;
  for (int i = 0; i < nw; ++i) {
    ss += s_sum[i];
    m = s_max[i] > m ? s_max[i] : m;
  }
  const float rstd = rstd_of(ss, a.V * 8, a.eps);
  const uint32_t am = magnitude_bits(__uint_as_float(m) * rstd);
  const float s8 = int8_scale(am), inv8 = 1.0f / s8;
  if (a.quant == kQuantInt8 && tid == 0) a.scales[row] = s8;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int32_t v = tid + i * blockDim.x;
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

// Threads and vectors a thread for rows of V vectors (V <= 4096).
static void row_shape(int32_t V, int &threads, int &vpt) {
  threads = V <= 64 ? 64 : V <= 128 ? 128 : V <= 1024 ? 256 : V <= 2048 ? 512 : 1024;
  const int n = (V + threads - 1) / threads;
  vpt = n <= 1 ? 1 : n <= 2 ? 2 : 4;
}

hipError_t launch_add_rmsnorm(const RmsNorm &n, hipStream_t s) {
  if (n.T == 0) return hipSuccess;
  const NormArgs a{reinterpret_cast<const u32x4 *>(n.x), n.residual, n.w, n.hidden,
                   reinterpret_cast<u32x4 *>(n.y), reinterpret_cast<u32x2 *>(n.codes), n.scales,
                   n.T, n.H / 8, n.w_fp32 ? 1 : 0, n.quant, n.eps};
  int threads, vpt;
  row_shape(a.V, threads, vpt);
#define L2(RT, RES, P) \
  hipLaunchKernelGGL((k_add_rmsnorm<RT, RES, P>), row_grid(n.T), dim3(threads), 0, s, a)
#define L(RT, RES)                  \
  do {                              \
    if (vpt == 1) L2(RT, RES, 1);   \
    else if (vpt == 2) L2(RT, RES, 2); \
    else L2(RT, RES, 4);            \
  } while (0)
  if (!n.residual) L(uint16_t, false);
  else if (n.res_fp32) L(float, true);
  else L(uint16_t, true);
#undef L
#undef L2
  return hipGetLastError();
}

// ---------------------------------------------------------------------------
// backward
//
// With n = h * rstd and g = grad_y * w:
//   grad_h = rstd * (g - n * mean(g * n)) [+ grad_hidden]
//   grad_w = sum over rows of grad_y * n
// One reduction over a row gives sum h^2 and sum g * h.  A workgroup takes
// every G-th row and keeps its share of grad_w in registers; the G partial
// rows go to the workspace and a second kernel adds them in order, in fp64, so
// the result does not depend on scheduling.

constexpr int32_t kNormBwdGroups = 512;

int32_t norm_bwd_groups(int32_t T) { return T < kNormBwdGroups ? T : kNormBwdGroups; }

struct NormBwdArgs {
  const void *hidden;
  const void *w;
  const u32x4 *gy;
  const void *ghidden;  // or null
  void *gx;
  float *part;          // [G][H] partial grad_w, or null
  int32_t T, V, w_fp32;
  double eps;
};

template <typename RT, int VPT>
__global__ __launch_bounds__(1024) void k_rmsnorm_bwd(NormBwdArgs a) {
  __shared__ double s_sum[2][16][2];
  const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6, nw = blockDim.x >> 6;
  float w[VPT][8], dw[VPT][8];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int32_t v = tid + i * blockDim.x;
#pragma unroll
    for (int c = 0; c < 8; ++c) w[i][c] = dw[i][c] = 0.0f;
    if (v < a.V) load_weight8(a.w, a.w_fp32, v, w[i]);
  }
  int buf = 0;
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x, buf ^= 1) {
    const int64_t base = t * a.V;
    float h[VPT][8], g[VPT][8];
    double ss = 0.0, sg = 0.0;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int32_t v = tid + i * blockDim.x;
#pragma unroll
      for (int c = 0; c < 8; ++c) h[i][c] = g[i][c] = 0.0f;
      if (v >= a.V) continue;
      load8<RT>(a.hidden, base + v, h[i]);
      unpack8(a.gy[base + v], g[i]);
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        ss += (double)h[i][c] * (double)h[i][c];
        sg += (double)(g[i][c] * w[i][c]) * (double)h[i][c];
      }
    }
    ss = wave_sum(ss);
    sg = wave_sum(sg);
    if (lane == 0) {
      s_sum[buf][wv][0] = ss;
      s_sum[buf][wv][1] = sg;
    }
    __syncthreads();   // two buffers: the next row's sums do not meet this row's readers
    ss = sg = 0.0;
    for (int i = 0; i < nw; ++i) {
      ss += s_sum[buf][i][0];
      sg += s_sum[buf][i][1];
    }
    const float rstd = rstd_of(ss, a.V * 8, a.eps);
    const float mean = (float)(sg * (double)rstd / (double)(a.V * 8));  // mean of g * n
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int32_t v = tid + i * blockDim.x;
      if (v >= a.V) continue;
      float o[8], r[8];
      if (a.ghidden) load8<RT>(a.ghidden, base + v, r);
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        const float n = h[i][c] * rstd;
        o[c] = rstd * (g[i][c] * w[i][c] - n * mean);
        if (a.ghidden) o[c] += r[c];
        dw[i][c] += g[i][c] * n;
      }
      store8<RT>(a.gx, base + v, o);
    }
  }
  if (a.part) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int32_t v = tid + i * blockDim.x;
      if (v < a.V) store8<float>(a.part, (int64_t)blockIdx.x * a.V + v, dw[i]);
    }
  }
}

__global__ __launch_bounds__(256) void k_rmsnorm_dw(const float *__restrict__ part, int32_t G,
                                                    int32_t H, float *__restrict__ dw) {
  const int32_t c = blockIdx.x * 256 + threadIdx.x;
  if (c >= H) return;
  double s = 0.0;
  for (int32_t i = 0; i < G; ++i) s += (double)part[(int64_t)i * H + c];
  dw[c] = (float)s;
}

hipError_t launch_rmsnorm_bwd(const RmsNormBwd &n, hipStream_t s) {
  if (n.T > 0) {
    const NormBwdArgs a{n.hidden, n.w, reinterpret_cast<const u32x4 *>(n.gy), n.ghidden, n.gx,
                        n.gw ? n.part : nullptr, n.T, n.H / 8, n.w_fp32 ? 1 : 0, n.eps};
    int threads, vpt;
    row_shape(a.V, threads, vpt);
    const unsigned G = (unsigned)norm_bwd_groups(n.T);
#define L2(RT, P) hipLaunchKernelGGL((k_rmsnorm_bwd<RT, P>), dim3(G), dim3(threads), 0, s, a)
#define L(RT)                    \
  do {                           \
    if (vpt == 1) L2(RT, 1);     \
    else if (vpt == 2) L2(RT, 2); \
    else L2(RT, 4);              \
  } while (0)
    if (n.h_fp32) L(float);
    else L(uint16_t);
#undef L
#undef L2
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (!n.gw) return hipSuccess;
  hipLaunchKernelGGL(k_rmsnorm_dw, dim3((unsigned)((n.H + 255) / 256)), dim3(256), 0, s, n.part,
                     norm_bwd_groups(n.T), n.H, n.gw);   // T == 0: zeros
  return hipGetLastError();
}

// ---------------------------------------------------------------------------
// INT8 rows from bf16 rows (the activation between an expert FFN's two INT8
// products): one workgroup per row, the row in registers between the
// reduction of its amax and its codes.

template <int VPT>
__global__ __launch_bounds__(1024) void k_quantize_int8(const u32x4 *__restrict__ x,
                                                        u32x2 *__restrict__ codes,
                                                        float *__restrict__ scales, int64_t rows,
                                                        int32_t V) {
  __shared__ uint32_t s_max[16];
  const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6, nw = blockDim.x >> 6;
  const int64_t row = grid_row(), base = row * V;
  if (row >= rows) return;
  float f[VPT][8];
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int32_t v = tid + i * blockDim.x;
    if (v >= V) continue;
    unpack8(x[base + v], f[i]);
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      const uint32_t b = magnitude_bits(f[i][c]);
      m = b > m ? b : m;
    }
  }
  m = wave_max(m);
  if (lane == 0) s_max[wv] = m;
  __syncthreads();
  m = 0;
  for (int i = 0; i < nw; ++i) m = s_max[i] > m ? s_max[i] : m;
  const float s = int8_scale(m), inv = 1.0f / s;
  if (tid == 0) scales[row] = s;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int32_t v = tid + i * blockDim.x;
    if (v < V) codes[base + v] = m >= kInfBits ? u32x2{0u, 0u} : int8_codes(f[i], s, inv);
  }
}

hipError_t launch_quantize_int8(const uint16_t *x, int64_t rows, int32_t K, uint8_t *codes,
                                float *scales, hipStream_t s) {
  if (rows == 0) return hipSuccess;
  const int32_t V = K / 8;
  int threads, vpt;
  row_shape(V, threads, vpt);
#define L(P)                                                                              \
  hipLaunchKernelGGL((k_quantize_int8<P>), row_grid(rows), dim3(threads), 0, s,           \
                     reinterpret_cast<const u32x4 *>(x), reinterpret_cast<u32x2 *>(codes), \
                     scales, rows, V)
  if (vpt == 1) L(1);
  else if (vpt == 2) L(2);
  else L(4);
#undef L
  return hipGetLastError();
}

}  // namespace epk
