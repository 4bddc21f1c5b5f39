// gemm_common.h -- what the grouped GEMM kernels share (gemm.hip: bf16 and FP8;
// gemm_int8.hip: INT8): tile sizes, the LDS chunk swizzle, the workgroup order
// over the tile table, loads that land in LDS.  gemm.hip describes the design.
#pragma once

#include "device.h"
#include "ep_internal.h"

namespace epk {

constexpr int kTileM = kGemmBM;
constexpr int kBN = 128;
constexpr int kWavesM = 2, kWavesN = 2;
constexpr int kGemmThreads = 64 * kWavesM * kWavesN;
constexpr int kWTM = kTileM / kWavesM, kWTN = kBN / kWavesN;  // one wave's output block
constexpr int kFM = kWTM / 32, kFN = kWTN / 32;                // 32 x 32 MFMA blocks per wave
constexpr int kBK = 64;
constexpr int kChunks = kBK / 8;  // 16-byte chunks in one row of a slab
constexpr int kXcds = 8;

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

__device__ __forceinline__ int swz(int row, int c) { return row * kChunks + (c ^ ((row >> 1) & 7)); }
static_assert(kChunks == 8, "the swizzle assumes 128-byte slab rows");

// 256 x 256 tiles
constexpr int kBM2 = 256, kBN2 = 256;                     // tile
constexpr int kWTM2 = kBM2 / 2, kWTN2 = kBN2 / 2;         // one wave's block (2 x 2 waves)
constexpr int kFM2 = kWTM2 / 32, kFN2 = kWTN2 / 32;       // 4 x 4 MFMA accumulators per wave
constexpr int kLoads2 = kBM2 * kChunks / kGemmThreads;    // 16-byte loads per thread per slab of X
constexpr int kLoadsB2 = kBN2 * kChunks / kGemmThreads;   // ... and of W
constexpr int kSlabA2 = kBM2 * kChunks, kSlabB2 = kBN2 * kChunks;
constexpr int kBufDword3 = 0x00020000;                    // buffer resource word 3 (raw, 32-bit data)

// What a kernel reads of the current plan's groups.
struct TileArgs {
  Geometry g;
  Workspace ws;
  int32_t use_slots;  // STATIC segments with a slot read weights from the slot
};

// Group q of the current plan: first receive row, rows, weight index
// (< E: owner expert; E + r*S + s: slot s of rank r).
__device__ __forceinline__ void group_of(const TileArgs &a, int32_t q, int32_t &row0,
                                         int32_t &rows, int32_t &widx) {
  const Geometry &g = a.g;
  const Workspace &ws = a.ws;
  if (g.layout == kHT) {
    row0 = ws.offsets[q];
    rows = ws.offsets[q + 1] - row0;
    widx = q;
  } else if (g.layout == kLL) {
    const int32_t c = ws.counts[q];
    row0 = q * g.cap;
    rows = c < g.cap ? c : g.cap;
    widx = q;
  } else if (q < g.E) {  // kept rows of expert q on its home rank
    const int32_t m = g.E / g.R;
    row0 = (q / m) * g.C + ws.native_row[q];
    rows = ws.keep[q];
    widx = q;
  } else {  // segment q - E on its receiving rank
    const int32_t *s = ws.segments + (int64_t)(q - g.E) * 5;
    const int32_t slot = ws.seg_slot[q - g.E];
    row0 = s[1] * g.C + s[4];
    rows = s[3];
    widx = (a.use_slots && slot >= 0) ? g.E + s[1] * g.S + slot : s[0];
  }
}

// Work of workgroup blockIdx.x: its row tile (an index into the table) and
// column tile.  Workgroup b runs on XCD b % 8; XCD x takes full tiles x,
// x + 8, x + 16, ... and short tiles x, x + 8, ..., each in group order,
// merged in proportion (Bresenham), every row tile with its column tiles one
// after another.  So every XCD gets the same MFMA-bound and streaming-bound
// work and runs both kinds side by side; the column tiles of a row tile stay
// on one XCD (they share X rows in its L2); and the eight XCDs walk the
// groups together, so the row tiles of one expert run on all of them at about
// the same time and its weight slices, after the first read, come from the
// Infinity Cache that the XCDs share (with each XCD taking a contiguous
// eighth, the row tiles of a hot expert ran one after another on one XCD and
// read its weights from HBM again each time).  The grid holds at least
// (max_tiles / 8 + 2) * n_col_tiles workgroups per XCD (gemm_grid).
__device__ __forceinline__ bool balanced_tile(const int32_t *__restrict__ ntiles,
                                              int32_t max_tiles, int32_t n_col_tiles,
                                              int32_t &tile, int32_t &col) {
  const int32_t nf = ntiles[1], ns = ntiles[0] - nf;
  const int32_t x = blockIdx.x % kXcds, slot = blockIdx.x / kXcds;
  // this XCD's full and short tiles: those whose index is x modulo 8
  const int32_t b = x < nf ? (nf - x + kXcds - 1) / kXcds : 0;
  const int32_t n = b + (x < ns ? (ns - x + kXcds - 1) / kXcds : 0);
  const int32_t p = slot / n_col_tiles;
  if (p >= n) return false;
  col = slot - p * n_col_tiles;
  const int32_t before = (int32_t)((int64_t)p * b / n), upto = (int32_t)((int64_t)(p + 1) * b / n);
  tile = upto > before ? x + kXcds * before : max_tiles - 1 - (x + kXcds * (p - before));
  return true;
}

#define LDS_PTR(p) ((__attribute__((address_space(3))) void *)(p))

// A buffer load whose lanes' 16 (or 4) bytes land in LDS at m0 + lane * 16
// (or 4), m0 being the wave's LDS base.  Written in asm on purpose: the
// compiler tracks its own form of this load and, unable to tell which part
// of LDS it writes, makes every later LDS read wait until it has landed --
// which would let no slab load run under the MFMAs of the previous slab.
// Here the caller owns the waits (s_waitcnt vmcnt before the barrier that
// publishes the data).  No result register: nothing the compiler allocates
// is written late.  The s_nop is the wait state the hardware needs between
// the write of m0 and the load that reads it.
__device__ __forceinline__ void lds_load16(__amdgpu_buffer_rsrc_t rsrc, uint32_t lds_base,
                                           uint32_t voff, uint32_t soff) {
  asm volatile("s_nop 0\n\tbuffer_load_dwordx4 %0, %1, %2 offen lds"
               :: "v"(voff), "s"(rsrc), "s"(soff), "{m0}"(lds_base) : "memory");
}
// ... of bytes nobody reads again soon: they do not displace what the caches hold.
__device__ __forceinline__ void lds_load16_stream(__amdgpu_buffer_rsrc_t rsrc, uint32_t lds_base,
                                                  uint32_t voff, uint32_t soff) {
  asm volatile("s_nop 0\n\tbuffer_load_dwordx4 %0, %1, %2 offen nt lds"
               :: "v"(voff), "s"(rsrc), "s"(soff), "{m0}"(lds_base) : "memory");
}
__device__ __forceinline__ void lds_load4(__amdgpu_buffer_rsrc_t rsrc, uint32_t lds_base,
                                          uint32_t voff, uint32_t soff) {
  asm volatile("s_nop 0\n\tbuffer_load_dword %0, %1, %2 offen lds"
               :: "v"(voff), "s"(rsrc), "s"(soff), "{m0}"(lds_base) : "memory");
}

// Workgroups of a GEMM launch: per XCD, room for an eighth of each kind of
// row tile rounded up (at most max_tiles / 8 + 2 row tiles), times the
// column tiles (balanced_tile).
inline int64_t gemm_grid_blocks(int32_t max_tiles, int32_t ncol) {
  return (int64_t)kXcds * (max_tiles / kXcds + 2) * ncol;
}

// Groups a plan can have (those of the current one are counted on the device).
inline int64_t gemm_groups(const Geometry &g) {
  return g.layout == kStatic ? 2 * (int64_t)g.E + g.R : g.E;
}

// At most as many 256-row tiles as the table holds 128-row ones.
inline int32_t wide_max_tiles(const Geometry &g) {
  const int64_t groups = gemm_groups(g);
  return (int32_t)((g.n + kBM2 - 1) / kBM2 + groups);
}

// Tile table of the current plan into ws.gemm_tiles / ws.gemm_ntiles: 256-row
// tiles, those of at most short_rows rows apart from the others, or (0)
// 128-row ones.
hipError_t launch_gemm_tiles(const Geometry &g, const Workspace &ws, bool slots,
                             int32_t short_rows, int32_t max_tiles, hipStream_t s);

}  // namespace epk
