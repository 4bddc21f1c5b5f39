// dropout.hip -- dropout of a layer's branch, joined with the residual stream
// (philox.h has the generator), on gfx950.
//
//   out = round(kept(x) * scale + residual)      (0 for what is dropped)
//
// The product and the sum are one fma, rounded to fp32 and then to out's type.
// The backward is the same call on the gradient, without a residual.  Bound by
// memory: each value is read and written once, vectors of eight, which are the
// generator's blocks (16384 x 4096 bf16 with a residual 61 us, 6.5 TB/s).
#include "ep_internal.h"
#include "philox.h"
#include "rows.h"

namespace epk {

// a value that stays times the scale, plus r; a dropped one gives r whatever it was
__device__ __forceinline__ float drop_add(float x, bool stay, float scale, float r) {
  return stay ? __builtin_fmaf(x, scale, r) : r;
}

constexpr int kDropThreads = 256;

template <typename XT, typename OT, bool RES>
__global__ __launch_bounds__(kDropThreads) void k_dropout(const void *x, const void *residual,
                                                          void *out, int64_t nvec, Dropout d) {
  const PhiloxKey key = philox_key(d.rng);
  const int64_t step = (int64_t)gridDim.x * kDropThreads;
  for (int64_t v = (int64_t)blockIdx.x * kDropThreads + threadIdx.x; v < nvec; v += step) {
    const Raw8<XT> xr = load_raw<XT, true>(x, v);
    Raw8<OT> rr;
    if constexpr (RES) rr = load_raw<OT, true>(residual, v);
    const u32x4 bits = philox((uint64_t)v, key);
    float f[8], r[8];
    unpack_raw(xr, f);
    if constexpr (RES) unpack_raw(rr, r);
#pragma unroll
    for (int c = 0; c < 8; ++c) f[c] = drop_add(f[c], stays(bits, c, d.threshold), d.scale, RES ? r[c] : 0.0f);
    store8<OT>(out, v, f);
  }
}

hipError_t launch_dropout(const DropoutAdd &n, hipStream_t s) {
  if (n.count == 0) return hipSuccess;
  const int64_t nvec = n.count / 8;
  const int64_t blocks = (nvec + kDropThreads - 1) / kDropThreads;
  const dim3 grid((unsigned)(blocks < 8192 ? blocks : 8192)), threads(kDropThreads);
#define L(XT, OT, RES) \
  hipLaunchKernelGGL((k_dropout<XT, OT, RES>), grid, threads, 0, s, n.x, n.residual, n.out, nvec, n.drop)
#define LR(XT, OT)                      \
  do {                                  \
    if (n.residual) L(XT, OT, true);    \
    else L(XT, OT, false);              \
  } while (0)
  if (n.x_fp32 && n.out_fp32) LR(float, float);
  else if (n.x_fp32) LR(float, uint16_t);
  else if (n.out_fp32) LR(uint16_t, float);
  else LR(uint16_t, uint16_t);
#undef LR
#undef L
  return hipGetLastError();
}

}  // namespace epk
