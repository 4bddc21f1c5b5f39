// dispatch8.hip -- token rows that are 8 bits already (INT8 codes with one
// fp32 scale a row, or FP8 codes with one per 128 channels) to their receive
// rows on gfx950, codes and scales bit for bit (see dispatch.hip for the
// layouts).  For rows a norm quantised: they are read at half the bytes of
// bf16 and quantised once instead of once per copy.
//
// Copies: every row is read once and written k times, so the kernel is bound
// by its writes.  One workgroup per token (per piece of a row for small
// batches), 16-byte loads and stores; the stores cached or non-temporal by the
// group's dispatch_stores, as in dispatch.hip.  Prefill (4096 x 7168, top-8):
// INT8 rows 52 us with cached stores where successive calls write other buffers,
// 40 where they write the same one (its lines are still in the Infinity Cache),
// 46 streaming; FP8 rows 59, 42 and 46.  With the INT8 GEMM behind it the pair is
// 0-2% faster cached, so that is the default at this size.
#include "device.h"
#include "ep_internal.h"

namespace epk {

constexpr int kRow8Threads = 512;

// Non-temporal stores?  The group's choice, or by size: cached between 64 MiB
// and 512 MiB of rows, counting those of every pass in flight against the upper
// bound (the rule ep_dispatch follows, on these rows' bytes).
static bool streaming_rows8(const Geometry &g, int64_t bytes) {
  if (g.stores != 0) return g.stores == 2;
  return bytes <= ((int64_t)64 << 20) || bytes * g.in_flight > ((int64_t)512 << 20);
}

template <int K, bool NT>
__global__ __launch_bounds__(kRow8Threads) void k_dispatch_rows8(
    const u32x4 *__restrict__ x, const float *__restrict__ xs, const int32_t *__restrict__ dst,
    u32x4 *__restrict__ recv, float *__restrict__ recv_s, int64_t rows, int32_t V, int32_t S,
    int32_t kr, int32_t chunk) {
  constexpr int KN = K > 0 ? K : kMaxTopK;
  const int64_t t = blockIdx.x;
  const int32_t k = K > 0 ? K : kr;
  const int32_t lo = blockIdx.y * chunk;
  const int32_t hi = lo + chunk < V ? lo + chunk : V;
  int32_t d[KN];
#pragma unroll
  for (int j = 0; j < KN; ++j) {
    const int32_t r = (K > 0 || j < k) ? dst[t * k + j] : -1;
    d[j] = r < rows ? r : -1;
  }
  for (int32_t v = lo + (int32_t)threadIdx.x; v < hi; v += kRow8Threads) {
    const u32x4 val = x[t * V + v];
#pragma unroll
    for (int j = 0; j < KN; ++j)
      if (d[j] >= 0) {
        if constexpr (NT) store_stream(recv + (int64_t)d[j] * V + v, val);
        else recv[(int64_t)d[j] * V + v] = val;
      }
  }
  if (blockIdx.y == 0) {
    for (int32_t i = threadIdx.x; i < S; i += kRow8Threads) {
      const float s = xs[t * S + i];
#pragma unroll
      for (int j = 0; j < KN; ++j)
        if (d[j] >= 0) recv_s[(int64_t)d[j] * S + i] = s;
    }
  }
}

hipError_t launch_dispatch_rows8(const Geometry &g, const Workspace &ws, const uint8_t *x,
                                 const float *xs, int32_t H, int32_t S, uint8_t *recv,
                                 float *recv_s, hipStream_t s) {
  if (g.T == 0) return hipSuccess;
  const int32_t V = H / 16;
  int32_t chunk = V;
  const int32_t pieces = row_pieces(g.T, V, &chunk);
  const bool nt = streaming_rows8(g, g.n * (H + 4 * (int64_t)S));
#define L2(KK, NT)                                                                          \
  hipLaunchKernelGGL((k_dispatch_rows8<KK, NT>), dim3((unsigned)g.T, pieces),               \
                     dim3(kRow8Threads), 0, s, reinterpret_cast<const u32x4 *>(x), xs, ws.dst, \
                     reinterpret_cast<u32x4 *>(recv), recv_s, g.rows, V, S, g.k, chunk)
#define L(KK)             \
  do {                    \
    if (nt) L2(KK, true); \
    else L2(KK, false);   \
  } while (0)
  EP_K_SWITCH(g.k, L)
#undef L
#undef L2
  return hipGetLastError();
}

}  // namespace epk
