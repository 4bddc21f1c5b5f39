// ep_api.cpp -- the C ABI declared in include/ep.h: argument validation,
// group and handle bookkeeping, workspace carving and kernel selection.
// Every check happens on the host before anything is enqueued; the only
// HIP calls are the kernel launches and, in ep_handle_status, one copy and
// one stream synchronisation.
#include <hip/hip_runtime.h>

#include <cfloat>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <new>

#include "ep.h"
#include "ep_internal.h"

struct ep_group {
  ep_group_config_t cfg;
  int32_t nbits;
};

struct ep_handle {
  ep_group *g;
  epk::Geometry geo;
  epk::Workspace ws;
  char *base;
  size_t bytes;
  bool planned;
  bool in_scratch;  // made by ep_handle_create_static: static storage, library scratch
};

namespace {
// The handles ep_handle_create_static returns: one per device, in static
// storage, so making one allocates nothing on the host either.
constexpr int kMaxScratchHandles = 64;
ep_handle g_scratch_handles[kMaxScratchHandles];
}  // namespace

namespace {

constexpr size_t kAlign = 256;
constexpr int64_t kFp8GemmMaxK = (int64_t)1 << 24;  // bytes per row of an FP8 GEMM operand

size_t align_up(size_t v) { return (v + kAlign - 1) & ~(kAlign - 1); }

epk::Geometry make_geometry(const ep_group *g, int32_t T) {
  const ep_group_config_t &c = g->cfg;
  epk::Geometry geo{};
  geo.T = T;
  geo.k = c.top_k;
  geo.E = c.num_experts;
  geo.R = c.num_ranks;
  geo.S = c.slots_per_rank;
  geo.slot_mode = c.slot_mode;
  geo.stores = c.dispatch_stores;
  geo.in_flight = c.passes_in_flight > 1 ? c.passes_in_flight : 1;
  geo.cstores = c.combine_stores;
  geo.fp8_pow2 = c.fp8_scales;   // 0 AMAX, 1 POW2, 2 AMAX rows with POW2 weights
  geo.layout = c.layout;
  geo.cap = c.capacity;
  geo.n = (int64_t)T * c.top_k;
  geo.C = (int32_t)((geo.n + c.num_ranks - 1) / c.num_ranks);
  const int64_t tiles = (geo.n + epk::kTileEntries - 1) / epk::kTileEntries;
  geo.ntiles = (int32_t)(tiles > 0 ? tiles : 1);
  geo.nbits = g->nbits;
  if (c.layout == EP_LAYOUT_HT) geo.rows = geo.n;
  else if (c.layout == EP_LAYOUT_LL) geo.rows = (int64_t)c.num_experts * c.capacity;
  else geo.rows = (int64_t)c.num_ranks * geo.C;
  return geo;
}

int64_t numel(const ep_tensor_t *t) {
  int64_t n = 1;
  for (int i = 0; i < t->ndim; ++i) n *= t->sizes[i];
  return n;
}

// Generic checks: non-NULL, tag, dtype, ndim in 1..4, sizes >= 0, data set and aligned.
ep_status_t check_tensor(const ep_tensor_t *t, int32_t tag, int32_t dtype) {
  if (!t) return EP_ERR_INVALID_ARG;
  if (t->tag != tag) return EP_ERR_BAD_TAG;
  if (t->dtype != dtype) return EP_ERR_BAD_DTYPE;
  if (t->ndim < 1 || t->ndim > 4 || t->reserved != 0) return EP_ERR_BAD_SHAPE;
  for (int i = 0; i < t->ndim; ++i)
    if (t->sizes[i] < 0) return EP_ERR_BAD_SHAPE;
  if (!t->data && numel(t) > 0) return EP_ERR_INVALID_ARG;
  // rows of tokens, expert weights and gradients move as 16-byte vectors;
  // ids, router weights, logits and scales as 4-byte words
  const uintptr_t need =
      (tag == EP_TAG_TOKENS || tag == EP_TAG_EXPERT_WEIGHTS || tag == EP_TAG_EXPERT_GRADS ||
       tag == EP_TAG_NORM_WEIGHT || tag == EP_TAG_WORKSPACE) ? 16 : 4;
  if (reinterpret_cast<uintptr_t>(t->data) % need != 0) return EP_ERR_INVALID_ARG;
  return EP_OK;
}

// Exactly [d0, d1] as a 2D tensor.
bool is_2d(const ep_tensor_t *t, int64_t d0, int64_t d1) {
  return t->ndim == 2 && t->sizes[0] == d0 && t->sizes[1] == d1;
}

// Leading sizes multiply to `rows`, last size `last` (any ndim >= 2), or a
// 1D tensor of `rows` elements when last == 1 and allow_1d.
bool is_rows(const ep_tensor_t *t, int64_t rows, int64_t last, bool allow_1d = false) {
  if (allow_1d && t->ndim == 1) return last == 1 && t->sizes[0] == rows;
  if (t->ndim < 2) return false;
  int64_t lead = 1;
  for (int i = 0; i + 1 < t->ndim; ++i) lead *= t->sizes[i];
  return lead == rows && t->sizes[t->ndim - 1] == last;
}

ep_status_t hip_status(hipError_t e) { return e == hipSuccess ? EP_OK : EP_ERR_HIP; }

// Compute units of the current device: a layout of at most that many tiles
// runs as one launch with every tile resident.  0 when there is no device (the
// layout then takes its two-launch form); a failed query's error is cleared
// so no later launch reports it.
int32_t device_cus() {
  int dev = 0, cus = 0;
  if (hipGetDevice(&dev) != hipSuccess ||
      hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess) {
    (void)hipGetLastError();
    return 0;
  }
  return cus;
}

hipStream_t as_stream(void *s) { return reinterpret_cast<hipStream_t>(s); }

}  // namespace

namespace epk {

size_t carve_workspace(const Geometry &g, char *base, Workspace *ws) {
  size_t off = 0;
  Workspace w{};
  auto take = [&](size_t bytes) -> char * {
    char *p = base ? base + off : nullptr;
    off += align_up(bytes > 0 ? bytes : 1);
    return p;
  };
  char *hdr = take(kAlign);
  w.status = reinterpret_cast<uint32_t *>(hdr);
  w.ticket = reinterpret_cast<uint32_t *>(hdr ? hdr + 4 : nullptr);
  w.stall = reinterpret_cast<uint32_t *>(hdr ? hdr + 8 : nullptr);
  w.arrive = reinterpret_cast<uint64_t *>(hdr ? hdr + 16 : nullptr);
  w.counts = reinterpret_cast<int32_t *>(take(sizeof(int32_t) * g.E));
  w.offsets = reinterpret_cast<int32_t *>(take(sizeof(int32_t) * (g.E + 1)));
  w.eidx = reinterpret_cast<int32_t *>(take(sizeof(int32_t) * g.n));
  w.lrank = reinterpret_cast<int32_t *>(take(sizeof(int32_t) * g.n));
  w.dst = reinterpret_cast<int32_t *>(take(sizeof(int32_t) * g.n));
  w.tile_hist = reinterpret_cast<int32_t *>(take(sizeof(int32_t) * (size_t)g.ntiles * g.E));
  w.tile_flags = reinterpret_cast<uint32_t *>(take(sizeof(uint32_t) * g.ntiles));
  w.tagged = reinterpret_cast<uint64_t *>(take(sizeof(uint64_t) * (size_t)g.ntiles * (g.E + 1)));
  w.recv_src = reinterpret_cast<int32_t *>(take(sizeof(int32_t) * g.rows));
  if (g.layout == kStatic) {
    w.keep = reinterpret_cast<int32_t *>(take(sizeof(int32_t) * g.E));
    w.native_row = reinterpret_cast<int32_t *>(take(sizeof(int32_t) * g.E));
    w.seg_first = reinterpret_cast<int32_t *>(take(sizeof(int32_t) * g.E));
    w.seg_count = reinterpret_cast<int32_t *>(take(sizeof(int32_t) * g.E));
    w.segments = reinterpret_cast<int32_t *>(take(sizeof(int32_t) * 5 * (size_t)(g.E + g.R)));
    w.n_segments = reinterpret_cast<int32_t *>(take(sizeof(int32_t)));
    w.load = reinterpret_cast<int32_t *>(take(sizeof(int32_t) * g.R));
    w.replica = reinterpret_cast<int32_t *>(take(sizeof(int32_t) * (size_t)g.R * g.S));
    w.seg_slot = reinterpret_cast<int32_t *>(take(sizeof(int32_t) * (size_t)(g.E + g.R)));
  }
  w.gemm_tiles = reinterpret_cast<int32_t *>(take(sizeof(int32_t) * 4 * (size_t)gemm_max_tiles(g)));
  w.gemm_ntiles = reinterpret_cast<int32_t *>(take(sizeof(int32_t) * 2));
  if (ws) *ws = w;
  return off;
}

}  // namespace epk

extern "C" {

const char *ep_status_string(ep_status_t st) {
  switch (st) {
    case EP_OK: return "EP_OK";
    case EP_ERR_INVALID_ARG: return "EP_ERR_INVALID_ARG";
    case EP_ERR_BAD_TAG: return "EP_ERR_BAD_TAG";
    case EP_ERR_BAD_DTYPE: return "EP_ERR_BAD_DTYPE";
    case EP_ERR_BAD_SHAPE: return "EP_ERR_BAD_SHAPE";
    case EP_ERR_NOT_PLANNED: return "EP_ERR_NOT_PLANNED";
    case EP_ERR_WORKSPACE_TOO_SMALL: return "EP_ERR_WORKSPACE_TOO_SMALL";
    case EP_ERR_UNSUPPORTED: return "EP_ERR_UNSUPPORTED";
    case EP_ERR_HIP: return "EP_ERR_HIP";
  }
  return "EP_ERR_UNKNOWN";
}

ep_status_t ep_group_create(const ep_group_config_t *cfg, ep_group_t *out) {
  if (!cfg || !out) return EP_ERR_INVALID_ARG;
  const ep_group_config_t &c = *cfg;
  if (c.num_experts < 1 || c.num_experts > epk::kMaxExperts) return EP_ERR_INVALID_ARG;
  if (c.num_ranks < 1 || c.num_experts % c.num_ranks != 0) return EP_ERR_INVALID_ARG;
  if (c.hidden < 8 || c.hidden % 8 != 0) return EP_ERR_INVALID_ARG;
  if (c.top_k < 1 || c.top_k > epk::kMaxTopK) return EP_ERR_INVALID_ARG;
  if (c.max_tokens < 0) return EP_ERR_INVALID_ARG;
  if ((int64_t)c.max_tokens * c.top_k > INT32_MAX) return EP_ERR_INVALID_ARG;
  if (c.layout != EP_LAYOUT_LL && c.layout != EP_LAYOUT_HT && c.layout != EP_LAYOUT_STATIC)
    return EP_ERR_INVALID_ARG;
  if (c.layout == EP_LAYOUT_LL &&
      (c.capacity < 1 || (int64_t)c.capacity * c.num_experts > INT32_MAX))
    return EP_ERR_INVALID_ARG;
  if (c.layout == EP_LAYOUT_STATIC &&
      (c.slots_per_rank < 0 || (int64_t)c.num_ranks * c.slots_per_rank > INT32_MAX))
    return EP_ERR_INVALID_ARG;
  if (c.dispatch_stores < EP_STORES_AUTO || c.dispatch_stores > EP_STORES_STREAMING)
    return EP_ERR_INVALID_ARG;
  if (c.passes_in_flight < 0 || c.passes_in_flight > 64) return EP_ERR_INVALID_ARG;
  if (c.combine_stores < EP_STORES_AUTO || c.combine_stores > EP_STORES_STREAMING)
    return EP_ERR_INVALID_ARG;
  if (c.fp8_scales != EP_FP8_SCALES_AMAX && c.fp8_scales != EP_FP8_SCALES_POW2 &&
      c.fp8_scales != EP_FP8_SCALES_AMAX_POW2_WEIGHTS)
    return EP_ERR_INVALID_ARG;
  if (c.slot_mode != EP_SLOTS_TRAINING &&
      !(c.slot_mode == EP_SLOTS_INFERENCE && c.layout == EP_LAYOUT_STATIC))
    return EP_ERR_INVALID_ARG;
  const int32_t R = c.layout == EP_LAYOUT_STATIC ? c.num_ranks : 0;
  if (epk::plan_lds_bytes(c.num_experts, R) + 256 > (size_t)epk::kLdsLimit)
    return EP_ERR_UNSUPPORTED;
  ep_group *g = new (std::nothrow) ep_group;
  if (!g) return EP_ERR_INVALID_ARG;
  g->cfg = c;
  g->nbits = 1;
  while ((1 << g->nbits) < c.num_experts) ++g->nbits;
  *out = g;
  return EP_OK;
}

ep_status_t ep_group_destroy(ep_group_t g) {
  if (!g) return EP_ERR_INVALID_ARG;
  delete g;
  return EP_OK;
}

ep_status_t ep_group_recv_rows(ep_group_t g, int32_t num_tokens, int64_t *rows) {
  if (!g || !rows || num_tokens < 0 || num_tokens > g->cfg.max_tokens) return EP_ERR_INVALID_ARG;
  *rows = make_geometry(g, num_tokens).rows;
  return EP_OK;
}

ep_status_t ep_handle_workspace_bytes(ep_group_t g, int32_t num_tokens, size_t *bytes) {
  if (!g || !bytes || num_tokens < 0 || num_tokens > g->cfg.max_tokens) return EP_ERR_INVALID_ARG;
  *bytes = epk::carve_workspace(make_geometry(g, num_tokens), nullptr, nullptr);
  return EP_OK;
}

ep_status_t ep_handle_create(ep_group_t g, int32_t num_tokens, void *workspace,
                             size_t workspace_bytes, ep_handle_t *out) {
  if (!g || !out || !workspace) return EP_ERR_INVALID_ARG;
  if (num_tokens < 0 || num_tokens > g->cfg.max_tokens) return EP_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(workspace) % kAlign != 0) return EP_ERR_INVALID_ARG;
  epk::Geometry geo = make_geometry(g, num_tokens);
  const size_t need = epk::carve_workspace(geo, nullptr, nullptr);
  if (workspace_bytes < need) return EP_ERR_WORKSPACE_TOO_SMALL;
  geo.cus = device_cus();
  ep_handle *h = new (std::nothrow) ep_handle;
  if (!h) return EP_ERR_INVALID_ARG;
  h->g = g;
  h->geo = geo;
  h->base = static_cast<char *>(workspace);
  h->bytes = workspace_bytes;
  h->planned = false;
  h->in_scratch = false;
  epk::carve_workspace(geo, h->base, &h->ws);
  *out = h;
  return EP_OK;
}

ep_status_t ep_handle_create_static(ep_group_t g, int32_t num_tokens, void *stream,
                                    ep_handle_t *out) {
  if (!g || !out) return EP_ERR_INVALID_ARG;
  if (num_tokens < 0 || num_tokens > g->cfg.max_tokens) return EP_ERR_INVALID_ARG;
  epk::Geometry geo = make_geometry(g, num_tokens);
  const size_t need = epk::carve_workspace(geo, nullptr, nullptr);
  if (need > epk::kScratchBytes) return EP_ERR_WORKSPACE_TOO_SMALL;
  int dev = 0;
  void *base = nullptr;
  if (epk::scratch_base(&dev, &base) != hipSuccess) {
    (void)hipGetLastError();
    return EP_ERR_HIP;
  }
  if (dev >= kMaxScratchHandles) return EP_ERR_UNSUPPORTED;
  // the workspace contract: zero-filled when the handle is made
  if (epk::launch_zero(base, need, as_stream(stream)) != hipSuccess) return EP_ERR_HIP;
  geo.cus = device_cus();
  ep_handle *h = &g_scratch_handles[dev];
  h->g = g;
  h->geo = geo;
  h->base = static_cast<char *>(base);
  h->bytes = epk::kScratchBytes;
  h->planned = false;
  h->in_scratch = true;
  epk::carve_workspace(geo, h->base, &h->ws);
  *out = h;
  return EP_OK;
}

ep_status_t ep_handle_destroy(ep_handle_t h) {
  if (!h) return EP_ERR_INVALID_ARG;
  if (h->in_scratch) return EP_OK;   // static storage: nothing to free
  delete h;
  return EP_OK;
}

ep_status_t ep_handle_query(ep_handle_t h, ep_handle_view_t *v) {
  if (!h || !v) return EP_ERR_INVALID_ARG;
  std::memset(v, 0, sizeof *v);
  const epk::Geometry &g = h->geo;
  v->num_tokens = g.T;
  v->top_k = g.k;
  v->num_experts = g.E;
  v->num_ranks = g.R;
  v->recv_rows = g.rows;
  v->rank_rows = g.layout == EP_LAYOUT_STATIC ? g.C
                 : g.layout == EP_LAYOUT_LL  ? g.cap
                                             : (int32_t)g.n;
  v->max_segments = g.layout == EP_LAYOUT_STATIC ? g.E + g.R : 0;
  v->counts = h->ws.counts;
  v->offsets = h->ws.offsets;
  v->dst = h->ws.dst;
  v->recv_src = h->ws.recv_src;
  v->status = h->ws.status;
  v->keep = h->ws.keep;
  v->native_row = h->ws.native_row;
  v->seg_first = h->ws.seg_first;
  v->seg_count = h->ws.seg_count;
  v->segments = h->ws.segments;
  v->n_segments = h->ws.n_segments;
  v->load = h->ws.load;
  v->replica = h->ws.replica;
  v->seg_slot = h->ws.seg_slot;
  return EP_OK;
}

ep_status_t ep_handle_status(ep_handle_t h, void *stream, uint32_t *flags) {
  if (!h || !flags) return EP_ERR_INVALID_ARG;
  // header: status word, ticket, stall mark, an unused word, arrival count
  uint32_t hdr[6] = {0, 0, 0, 0, 0, 0};
  hipError_t e = hipMemcpyAsync(hdr, h->ws.status, sizeof hdr, hipMemcpyDeviceToHost,
                                as_stream(stream));
  if (e == hipSuccess) e = hipStreamSynchronize(as_stream(stream));
  if (e != hipSuccess) return EP_ERR_HIP;
  uint32_t v = hdr[0];
  // resident-tiles layout: the last call's epoch mark is its calls so far
  const epk::Geometry &g = h->geo;
  if (g.ntiles > 1 && g.ntiles <= g.cus) {
    uint64_t arrive;
    std::memcpy(&arrive, hdr + 4, sizeof arrive);
    const uint32_t last = (uint32_t)(arrive / (uint64_t)g.ntiles);
    if (last != 0 && hdr[2] == last) v |= EP_FLAG_PLAN_STALL;
  }
  *flags = v;
  return EP_OK;
}

ep_status_t ep_route(ep_handle_t h, const ep_tensor_t *logits, ep_tensor_t *topk_idx,
                     ep_tensor_t *topk_weights, void *stream) {
  if (!h) return EP_ERR_INVALID_ARG;
  const epk::Geometry &g = h->geo;
  ep_status_t st = check_tensor(logits, EP_TAG_ROUTER_LOGITS, EP_DTYPE_FP32);
  if (st != EP_OK) return st;
  if (!is_2d(logits, g.T, g.E)) return EP_ERR_BAD_SHAPE;
  st = check_tensor(topk_idx, EP_TAG_TOPK_IDX, EP_DTYPE_INT32);
  if (st != EP_OK) return st;
  if (!is_2d(topk_idx, g.T, g.k)) return EP_ERR_BAD_SHAPE;
  st = check_tensor(topk_weights, EP_TAG_TOPK_WEIGHTS, EP_DTYPE_FP32);
  if (st != EP_OK) return st;
  if (!is_2d(topk_weights, g.T, g.k)) return EP_ERR_BAD_SHAPE;
  return hip_status(epk::launch_route(static_cast<const float *>(logits->data), g.T, g.E, g.k,
                                      static_cast<int32_t *>(topk_idx->data),
                                      static_cast<float *>(topk_weights->data),
                                      as_stream(stream)));
}

ep_status_t ep_route_plan(ep_handle_t h, const ep_tensor_t *logits, ep_tensor_t *topk_idx,
                          ep_tensor_t *topk_weights, void *stream) {
  if (!h) return EP_ERR_INVALID_ARG;
  const epk::Geometry &g = h->geo;
  ep_status_t st = check_tensor(logits, EP_TAG_ROUTER_LOGITS, EP_DTYPE_FP32);
  if (st != EP_OK) return st;
  if (!is_2d(logits, g.T, g.E)) return EP_ERR_BAD_SHAPE;
  st = check_tensor(topk_idx, EP_TAG_TOPK_IDX, EP_DTYPE_INT32);
  if (st != EP_OK) return st;
  if (!is_2d(topk_idx, g.T, g.k)) return EP_ERR_BAD_SHAPE;
  st = check_tensor(topk_weights, EP_TAG_TOPK_WEIGHTS, EP_DTYPE_FP32);
  if (st != EP_OK) return st;
  if (!is_2d(topk_weights, g.T, g.k)) return EP_ERR_BAD_SHAPE;
  st = hip_status(epk::launch_route_plan(g, h->ws, static_cast<const float *>(logits->data),
                                         static_cast<int32_t *>(topk_idx->data),
                                         static_cast<float *>(topk_weights->data),
                                         as_stream(stream)));
  if (st == EP_OK) h->planned = true;
  return st;
}

ep_status_t ep_plan(ep_handle_t h, const ep_tensor_t *topk_idx, void *stream) {
  if (!h) return EP_ERR_INVALID_ARG;
  const epk::Geometry &g = h->geo;
  ep_status_t st = check_tensor(topk_idx, EP_TAG_TOPK_IDX, EP_DTYPE_INT32);
  if (st != EP_OK) return st;
  if (!is_2d(topk_idx, g.T, g.k)) return EP_ERR_BAD_SHAPE;
  st = hip_status(epk::launch_plan(g, h->ws, static_cast<const int32_t *>(topk_idx->data),
                                   as_stream(stream)));
  if (st == EP_OK) h->planned = true;
  return st;
}

// The optional weights and per-row outputs of a dispatch.
static ep_status_t check_recv_meta(const epk::Geometry &g, const ep_tensor_t *topk_weights,
                                   const ep_tensor_t *recv_topk_idx,
                                   const ep_tensor_t *recv_topk_weights) {
  ep_status_t st;
  if (topk_weights) {
    st = check_tensor(topk_weights, EP_TAG_TOPK_WEIGHTS, EP_DTYPE_FP32);
    if (st != EP_OK) return st;
    if (!is_2d(topk_weights, g.T, g.k)) return EP_ERR_BAD_SHAPE;
  }
  if (recv_topk_idx) {
    st = check_tensor(recv_topk_idx, EP_TAG_TOPK_IDX, EP_DTYPE_INT32);
    if (st != EP_OK) return st;
    if (!(recv_topk_idx->ndim == 1 && recv_topk_idx->sizes[0] == g.rows)) return EP_ERR_BAD_SHAPE;
  }
  if (recv_topk_weights) {
    if (!topk_weights) return EP_ERR_INVALID_ARG;
    st = check_tensor(recv_topk_weights, EP_TAG_TOPK_WEIGHTS, EP_DTYPE_FP32);
    if (st != EP_OK) return st;
    if (!(recv_topk_weights->ndim == 1 && recv_topk_weights->sizes[0] == g.rows))
      return EP_ERR_BAD_SHAPE;
  }
  return EP_OK;
}

// Argument checks of a dispatch (tokens, optional weights, receive rows and
// scales, optional per-row outputs); EP_OK when all hold.
static ep_status_t check_dispatch(const ep_handle *h, const ep_tensor_t *tokens,
                                  const ep_tensor_t *topk_weights, const ep_tensor_t *recv_tokens,
                                  const ep_tensor_t *recv_scales, const ep_tensor_t *recv_topk_idx,
                                  const ep_tensor_t *recv_topk_weights) {
  const epk::Geometry &g = h->geo;
  const int32_t H = h->g->cfg.hidden;
  ep_status_t st = check_tensor(tokens, EP_TAG_TOKENS, EP_DTYPE_BF16);
  if (st != EP_OK) return st;
  if (!is_2d(tokens, g.T, H)) return EP_ERR_BAD_SHAPE;
  const bool fp8 = recv_scales != nullptr;
  st = check_tensor(recv_tokens, EP_TAG_TOKENS, fp8 ? EP_DTYPE_FP8_E4M3 : EP_DTYPE_BF16);
  if (st != EP_OK) return st;
  if (!is_rows(recv_tokens, g.rows, H)) return EP_ERR_BAD_SHAPE;
  if (fp8) {
    if (H % 128 != 0) return EP_ERR_UNSUPPORTED;
    st = check_tensor(recv_scales, EP_TAG_FP8_SCALES, EP_DTYPE_FP32);
    if (st != EP_OK) return st;
    if (!is_rows(recv_scales, g.rows, H / 128)) return EP_ERR_BAD_SHAPE;
  }
  return check_recv_meta(g, topk_weights, recv_topk_idx, recv_topk_weights);
}

// Enqueue a checked dispatch; fused: the layout of topk_idx in the same launch.
static ep_status_t run_dispatch(ep_handle *h, const ep_tensor_t *tokens,
                                const ep_tensor_t *topk_weights, ep_tensor_t *recv_tokens,
                                ep_tensor_t *recv_scales, ep_tensor_t *recv_topk_idx,
                                ep_tensor_t *recv_topk_weights, hipStream_t s,
                                const int32_t *topk_idx, bool fused) {
  const epk::Geometry &g = h->geo;
  const int32_t H = h->g->cfg.hidden;
  hipError_t e;
  if (recv_scales)
    e = epk::launch_dispatch_fp8(g, h->ws, static_cast<const uint16_t *>(tokens->data), H,
                                 static_cast<uint8_t *>(recv_tokens->data),
                                 static_cast<float *>(recv_scales->data), s, topk_idx, fused);
  else
    e = epk::launch_dispatch_bf16(g, h->ws, static_cast<const uint16_t *>(tokens->data), H,
                                  static_cast<uint16_t *>(recv_tokens->data), s, topk_idx, fused);
  if (e == hipSuccess && (recv_topk_idx || recv_topk_weights))
    e = epk::launch_recv_meta(
        g, h->ws, topk_weights ? static_cast<const float *>(topk_weights->data) : nullptr,
        recv_topk_idx ? static_cast<int32_t *>(recv_topk_idx->data) : nullptr,
        recv_topk_weights ? static_cast<float *>(recv_topk_weights->data) : nullptr, s);
  return hip_status(e);
}

ep_status_t ep_dispatch(ep_handle_t h, const ep_tensor_t *tokens, const ep_tensor_t *topk_weights,
                        ep_tensor_t *recv_tokens, ep_tensor_t *recv_scales,
                        ep_tensor_t *recv_topk_idx, ep_tensor_t *recv_topk_weights,
                        void *stream) {
  if (!h) return EP_ERR_INVALID_ARG;
  ep_status_t st = check_dispatch(h, tokens, topk_weights, recv_tokens, recv_scales,
                                  recv_topk_idx, recv_topk_weights);
  if (st != EP_OK) return st;
  if (!h->planned) return EP_ERR_NOT_PLANNED;
  return run_dispatch(h, tokens, topk_weights, recv_tokens, recv_scales, recv_topk_idx,
                      recv_topk_weights, as_stream(stream), nullptr, false);
}

ep_status_t ep_plan_dispatch(ep_handle_t h, const ep_tensor_t *topk_idx,
                             const ep_tensor_t *tokens, const ep_tensor_t *topk_weights,
                             ep_tensor_t *recv_tokens, ep_tensor_t *recv_scales,
                             ep_tensor_t *recv_topk_idx, ep_tensor_t *recv_topk_weights,
                             void *stream) {
  if (!h) return EP_ERR_INVALID_ARG;
  const epk::Geometry &g = h->geo;
  ep_status_t st = check_tensor(topk_idx, EP_TAG_TOPK_IDX, EP_DTYPE_INT32);
  if (st != EP_OK) return st;
  if (!is_2d(topk_idx, g.T, g.k)) return EP_ERR_BAD_SHAPE;
  st = check_dispatch(h, tokens, topk_weights, recv_tokens, recv_scales, recv_topk_idx,
                      recv_topk_weights);
  if (st != EP_OK) return st;
  hipStream_t s = as_stream(stream);
  const int32_t *idx = static_cast<const int32_t *>(topk_idx->data);
  const bool fused = epk::fused_layout_fits(g);
  if (!fused) {
    st = hip_status(epk::launch_plan(g, h->ws, idx, s));
    if (st != EP_OK) return st;
  }
  h->planned = true;
  return run_dispatch(h, tokens, topk_weights, recv_tokens, recv_scales, recv_topk_idx,
                      recv_topk_weights, s, idx, fused);
}

ep_status_t ep_quantize_fp8(const ep_tensor_t *tokens, ep_tensor_t *codes, ep_tensor_t *scales,
                            int32_t fp8_scales, void *stream) {
  if (fp8_scales != EP_FP8_SCALES_AMAX && fp8_scales != EP_FP8_SCALES_POW2) return EP_ERR_INVALID_ARG;
  ep_status_t st = check_tensor(tokens, EP_TAG_TOKENS, EP_DTYPE_BF16);
  if (st != EP_OK) return st;
  st = check_tensor(codes, EP_TAG_TOKENS, EP_DTYPE_FP8_E4M3);
  if (st != EP_OK) return st;
  st = check_tensor(scales, EP_TAG_FP8_SCALES, EP_DTYPE_FP32);
  if (st != EP_OK) return st;
  if (tokens->ndim < 2) return EP_ERR_BAD_SHAPE;
  const int64_t K = tokens->sizes[tokens->ndim - 1];
  const int64_t rows = numel(tokens) / (K > 0 ? K : 1);
  if (K <= 0 || K % 128 != 0 || K > INT32_MAX) return EP_ERR_BAD_SHAPE;
  if (!is_rows(codes, rows, K) || !is_rows(scales, rows, K / 128)) return EP_ERR_BAD_SHAPE;
  return hip_status(epk::launch_quantize_fp8(static_cast<const uint16_t *>(tokens->data), rows,
                                             (int32_t)K, static_cast<uint8_t *>(codes->data),
                                             static_cast<float *>(scales->data),
                                             fp8_scales == EP_FP8_SCALES_POW2, as_stream(stream)));
}

ep_status_t ep_combine(ep_handle_t h, const ep_tensor_t *expert_out,
                       const ep_tensor_t *topk_weights, ep_tensor_t *out_tokens, void *stream) {
  if (!h) return EP_ERR_INVALID_ARG;
  const epk::Geometry &g = h->geo;
  const int32_t H = h->g->cfg.hidden;
  ep_status_t st = check_tensor(expert_out, EP_TAG_TOKENS, EP_DTYPE_BF16);
  if (st != EP_OK) return st;
  if (!is_rows(expert_out, g.rows, H)) return EP_ERR_BAD_SHAPE;
  if (topk_weights) {
    st = check_tensor(topk_weights, EP_TAG_TOPK_WEIGHTS, EP_DTYPE_FP32);
    if (st != EP_OK) return st;
    if (!is_2d(topk_weights, g.T, g.k)) return EP_ERR_BAD_SHAPE;
  }
  if (!out_tokens) return EP_ERR_INVALID_ARG;
  const bool out_fp32 = out_tokens->dtype == EP_DTYPE_FP32;
  st = check_tensor(out_tokens, EP_TAG_TOKENS, out_fp32 ? EP_DTYPE_FP32 : EP_DTYPE_BF16);
  if (st != EP_OK) return st;
  if (!is_2d(out_tokens, g.T, H)) return EP_ERR_BAD_SHAPE;
  if (!h->planned) return EP_ERR_NOT_PLANNED;
  return hip_status(epk::launch_combine(
      g, h->ws, static_cast<const uint16_t *>(expert_out->data), H,
      topk_weights ? static_cast<const float *>(topk_weights->data) : nullptr, out_tokens->data,
      out_fp32, as_stream(stream)));
}

ep_status_t ep_combine_bwd(ep_handle_t h, const ep_tensor_t *grad_tokens,
                           const ep_tensor_t *expert_out, const ep_tensor_t *topk_weights,
                           ep_tensor_t *grad_expert_out, ep_tensor_t *grad_topk_weights,
                           void *stream) {
  if (!h) return EP_ERR_INVALID_ARG;
  const epk::Geometry &g = h->geo;
  const int32_t H = h->g->cfg.hidden;
  ep_status_t st = check_tensor(grad_tokens, EP_TAG_TOKENS, EP_DTYPE_BF16);
  if (st != EP_OK) return st;
  if (!is_2d(grad_tokens, g.T, H)) return EP_ERR_BAD_SHAPE;
  st = check_tensor(expert_out, EP_TAG_TOKENS, EP_DTYPE_BF16);
  if (st != EP_OK) return st;
  if (!is_rows(expert_out, g.rows, H)) return EP_ERR_BAD_SHAPE;
  st = check_tensor(topk_weights, EP_TAG_TOPK_WEIGHTS, EP_DTYPE_FP32);
  if (st != EP_OK) return st;
  if (!is_2d(topk_weights, g.T, g.k)) return EP_ERR_BAD_SHAPE;
  st = check_tensor(grad_expert_out, EP_TAG_TOKENS, EP_DTYPE_BF16);
  if (st != EP_OK) return st;
  if (!is_rows(grad_expert_out, g.rows, H)) return EP_ERR_BAD_SHAPE;
  st = check_tensor(grad_topk_weights, EP_TAG_TOPK_WEIGHTS, EP_DTYPE_FP32);
  if (st != EP_OK) return st;
  if (!is_2d(grad_topk_weights, g.T, g.k)) return EP_ERR_BAD_SHAPE;
  if (!h->planned) return EP_ERR_NOT_PLANNED;
  return hip_status(epk::launch_combine_bwd(
      g, h->ws, static_cast<const uint16_t *>(grad_tokens->data),
      static_cast<const uint16_t *>(expert_out->data), H,
      static_cast<const float *>(topk_weights->data),
      static_cast<uint16_t *>(grad_expert_out->data),
      static_cast<float *>(grad_topk_weights->data), as_stream(stream)));
}

ep_status_t ep_dup_grad_reduce(ep_handle_t h, const ep_tensor_t *replica_grads,
                               const ep_tensor_t *replica_expert, ep_tensor_t *owner_grads,
                               void *stream) {
  if (!h) return EP_ERR_INVALID_ARG;
  ep_status_t st = check_tensor(replica_grads, EP_TAG_EXPERT_GRADS, EP_DTYPE_BF16);
  if (st != EP_OK) return st;
  st = check_tensor(owner_grads, EP_TAG_EXPERT_GRADS, EP_DTYPE_FP32);
  if (st != EP_OK) return st;
  if (replica_grads->ndim < 2 || owner_grads->ndim < 2) return EP_ERR_BAD_SHAPE;
  const int64_t n = replica_grads->sizes[0];
  const int64_t P = numel(replica_grads) / (n > 0 ? n : 1);
  const int64_t E_owner = owner_grads->sizes[0];
  int64_t Po = 1;
  for (int i = 1; i < owner_grads->ndim; ++i) Po *= owner_grads->sizes[i];
  if (replica_grads->ndim != owner_grads->ndim) return EP_ERR_BAD_SHAPE;
  for (int i = 1; i < owner_grads->ndim; ++i)
    if (replica_grads->sizes[i] != owner_grads->sizes[i]) return EP_ERR_BAD_SHAPE;
  if (n > 65535 || E_owner > INT32_MAX || Po != P) return EP_ERR_BAD_SHAPE;
  const int32_t *rep_e = nullptr;
  if (replica_expert) {
    st = check_tensor(replica_expert, EP_TAG_TOPK_IDX, EP_DTYPE_INT32);
    if (st != EP_OK) return st;
    if (!(replica_expert->ndim == 1 && replica_expert->sizes[0] == n)) return EP_ERR_BAD_SHAPE;
    rep_e = static_cast<const int32_t *>(replica_expert->data);
  } else {
    if (h->geo.layout != EP_LAYOUT_STATIC) return EP_ERR_UNSUPPORTED;
    if (n != (int64_t)h->geo.R * h->geo.S) return EP_ERR_BAD_SHAPE;
    if (!h->planned) return EP_ERR_NOT_PLANNED;
    rep_e = h->ws.replica;
  }
  return hip_status(epk::launch_dup_reduce(
      static_cast<const uint16_t *>(replica_grads->data), rep_e, (int32_t)n, P, (int32_t)E_owner,
      static_cast<float *>(owner_grads->data), h->ws.status, as_stream(stream)));
}

ep_status_t ep_prefetch_replicas(ep_handle_t h, const ep_tensor_t *expert_weights,
                                 ep_tensor_t *slot_weights, void *stream) {
  if (!h || !expert_weights || !slot_weights) return EP_ERR_INVALID_ARG;
  const epk::Geometry &g = h->geo;
  const int32_t dt = expert_weights->dtype;
  // the weights themselves, or the fp32 scales of FP8 or INT8 weights
  const int32_t wt = expert_weights->tag;
  const bool scales = wt == EP_TAG_FP8_SCALES || wt == EP_TAG_ROW_SCALES;
  const int32_t tag = scales ? wt : EP_TAG_EXPERT_WEIGHTS;
  if (scales ? dt != EP_DTYPE_FP32
             : dt != EP_DTYPE_BF16 && dt != EP_DTYPE_FP32 && dt != EP_DTYPE_FP8_E4M3 &&
                   dt != EP_DTYPE_INT8)
    return EP_ERR_BAD_DTYPE;
  ep_status_t st = check_tensor(expert_weights, tag, dt);
  if (st != EP_OK) return st;
  st = check_tensor(slot_weights, tag, dt);
  if (st != EP_OK) return st;
  if (g.layout != EP_LAYOUT_STATIC) return EP_ERR_UNSUPPORTED;
  // expert_weights [E, P...]; slot_weights [R, S, P...] or [R*S, P...]
  const ep_tensor_t *w = expert_weights, *sl = slot_weights;
  if (w->ndim < 2 || w->sizes[0] != g.E) return EP_ERR_BAD_SHAPE;
  int64_t P = 1;
  for (int i = 1; i < w->ndim; ++i) P *= w->sizes[i];
  const int tail = w->ndim - 1;  // dims of one row
  if (sl->ndim == tail + 2) {
    if (sl->sizes[0] != g.R || sl->sizes[1] != g.S) return EP_ERR_BAD_SHAPE;
  } else if (sl->ndim == tail + 1) {
    if (sl->sizes[0] != (int64_t)g.R * g.S) return EP_ERR_BAD_SHAPE;
  } else {
    return EP_ERR_BAD_SHAPE;
  }
  for (int i = 0; i < tail; ++i)
    if (sl->sizes[sl->ndim - tail + i] != w->sizes[1 + i]) return EP_ERR_BAD_SHAPE;
  const int64_t elem = dt == EP_DTYPE_FP32 ? 4 : dt == EP_DTYPE_BF16 ? 2 : 1;
  const int64_t row_bytes = P * elem;
  if (row_bytes % 4 != 0) return EP_ERR_BAD_SHAPE;
  if (!h->planned) return EP_ERR_NOT_PLANNED;
  return hip_status(epk::launch_prefetch(g, h->ws, static_cast<const uint8_t *>(w->data),
                                         row_bytes, static_cast<uint8_t *>(sl->data),
                                         as_stream(stream)));
}

// glu: the SwiGLU epilogue (out has N / 2 columns; N % 16 == 0)
static ep_status_t expert_gemm(ep_handle_t h, const ep_tensor_t *recv_tokens,
                               const ep_tensor_t *expert_weights, const ep_tensor_t *slot_weights,
                               ep_tensor_t *out, void *stream, bool glu) {
  if (!h) return EP_ERR_INVALID_ARG;
  const epk::Geometry &g = h->geo;
  ep_status_t st = check_tensor(recv_tokens, EP_TAG_TOKENS, EP_DTYPE_BF16);
  if (st != EP_OK) return st;
  st = check_tensor(expert_weights, EP_TAG_EXPERT_WEIGHTS, EP_DTYPE_BF16);
  if (st != EP_OK) return st;
  st = check_tensor(out, EP_TAG_TOKENS, EP_DTYPE_BF16);
  if (st != EP_OK) return st;
  const ep_tensor_t *w = expert_weights;
  if (w->ndim != 3 || w->sizes[0] != g.E) return EP_ERR_BAD_SHAPE;
  const int64_t N = w->sizes[1], K = w->sizes[2];
  if (K <= 0 || K % 64 != 0 || K > INT32_MAX || N < 1 || N > INT32_MAX) return EP_ERR_BAD_SHAPE;
  if (glu && N % 16 != 0) return EP_ERR_BAD_SHAPE;
  if (!is_rows(recv_tokens, g.rows, K) || !is_rows(out, g.rows, glu ? N / 2 : N))
    return EP_ERR_BAD_SHAPE;
  const uint16_t *wslot = nullptr;
  if (slot_weights) {
    st = check_tensor(slot_weights, EP_TAG_EXPERT_WEIGHTS, EP_DTYPE_BF16);
    if (st != EP_OK) return st;
    if (g.layout != EP_LAYOUT_STATIC) return EP_ERR_UNSUPPORTED;
    const ep_tensor_t *sl = slot_weights;
    const bool four = sl->ndim == 4 && sl->sizes[0] == g.R && sl->sizes[1] == g.S &&
                      sl->sizes[2] == N && sl->sizes[3] == K;
    const bool three = sl->ndim == 3 && sl->sizes[0] == (int64_t)g.R * g.S && sl->sizes[1] == N &&
                       sl->sizes[2] == K;
    if (!four && !three) return EP_ERR_BAD_SHAPE;
    wslot = static_cast<const uint16_t *>(sl->data);
  }
  if (!h->planned) return EP_ERR_NOT_PLANNED;
  return hip_status(epk::launch_grouped_gemm(g, h->ws, static_cast<const uint16_t *>(recv_tokens->data),
                                             static_cast<const uint16_t *>(w->data), wslot,
                                             (int32_t)K, (int32_t)N,
                                             static_cast<uint16_t *>(out->data), glu,
                                             as_stream(stream)));
}

ep_status_t ep_expert_gemm(ep_handle_t h, const ep_tensor_t *recv_tokens,
                           const ep_tensor_t *expert_weights, const ep_tensor_t *slot_weights,
                           ep_tensor_t *out, void *stream) {
  return expert_gemm(h, recv_tokens, expert_weights, slot_weights, out, stream, false);
}

ep_status_t ep_expert_gemm_swiglu(ep_handle_t h, const ep_tensor_t *recv_tokens,
                                  const ep_tensor_t *expert_weights,
                                  const ep_tensor_t *slot_weights, ep_tensor_t *out,
                                  void *stream) {
  return expert_gemm(h, recv_tokens, expert_weights, slot_weights, out, stream, true);
}

static ep_status_t expert_gemm_fp8(ep_handle_t h, const ep_tensor_t *recv_tokens,
                                   const ep_tensor_t *recv_scales,
                                   const ep_tensor_t *expert_weights,
                                   const ep_tensor_t *expert_scales,
                                   const ep_tensor_t *slot_weights, const ep_tensor_t *slot_scales,
                                   ep_tensor_t *out, void *stream, bool glu) {
  if (!h) return EP_ERR_INVALID_ARG;
  const epk::Geometry &g = h->geo;
  ep_status_t st = check_tensor(recv_tokens, EP_TAG_TOKENS, EP_DTYPE_FP8_E4M3);
  if (st != EP_OK) return st;
  st = check_tensor(recv_scales, EP_TAG_FP8_SCALES, EP_DTYPE_FP32);
  if (st != EP_OK) return st;
  st = check_tensor(expert_weights, EP_TAG_EXPERT_WEIGHTS, EP_DTYPE_FP8_E4M3);
  if (st != EP_OK) return st;
  st = check_tensor(expert_scales, EP_TAG_FP8_SCALES, EP_DTYPE_FP32);
  if (st != EP_OK) return st;
  st = check_tensor(out, EP_TAG_TOKENS, EP_DTYPE_BF16);
  if (st != EP_OK) return st;
  const ep_tensor_t *w = expert_weights, *ws = expert_scales;
  if (w->ndim != 3 || w->sizes[0] != g.E) return EP_ERR_BAD_SHAPE;
  const int64_t N = w->sizes[1], K = w->sizes[2];
  if (K <= 0 || K % 128 != 0 || K > INT32_MAX || N < 1 || N > INT32_MAX) return EP_ERR_BAD_SHAPE;
  if (glu && N % 16 != 0) return EP_ERR_BAD_SHAPE;
  // the kernel addresses a tile's 128 rows of K bytes through 32-bit buffer offsets
  if (K > kFp8GemmMaxK) return EP_ERR_UNSUPPORTED;
  const int64_t NB = K / 128;
  if (!(ws->ndim == 3 && ws->sizes[0] == g.E && ws->sizes[1] == N && ws->sizes[2] == NB))
    return EP_ERR_BAD_SHAPE;
  if (!is_rows(recv_tokens, g.rows, K) || !is_rows(recv_scales, g.rows, NB) ||
      !is_rows(out, g.rows, glu ? N / 2 : N))
    return EP_ERR_BAD_SHAPE;
  if ((slot_weights == nullptr) != (slot_scales == nullptr)) return EP_ERR_INVALID_ARG;
  const uint8_t *wslot = nullptr;
  const float *swslot = nullptr;
  if (slot_weights) {
    st = check_tensor(slot_weights, EP_TAG_EXPERT_WEIGHTS, EP_DTYPE_FP8_E4M3);
    if (st != EP_OK) return st;
    st = check_tensor(slot_scales, EP_TAG_FP8_SCALES, EP_DTYPE_FP32);
    if (st != EP_OK) return st;
    if (g.layout != EP_LAYOUT_STATIC) return EP_ERR_UNSUPPORTED;
    const int64_t RS = (int64_t)g.R * g.S;
    auto slots_of = [&](const ep_tensor_t *t, int64_t last) {
      return (t->ndim == 4 && t->sizes[0] == g.R && t->sizes[1] == g.S && t->sizes[2] == N &&
              t->sizes[3] == last) ||
             (t->ndim == 3 && t->sizes[0] == RS && t->sizes[1] == N && t->sizes[2] == last);
    };
    if (!slots_of(slot_weights, K) || !slots_of(slot_scales, NB)) return EP_ERR_BAD_SHAPE;
    wslot = static_cast<const uint8_t *>(slot_weights->data);
    swslot = static_cast<const float *>(slot_scales->data);
  }
  if (!h->planned) return EP_ERR_NOT_PLANNED;
  return hip_status(epk::launch_grouped_gemm_fp8(
      g, h->ws, static_cast<const uint8_t *>(recv_tokens->data),
      static_cast<const float *>(recv_scales->data), static_cast<const uint8_t *>(w->data),
      static_cast<const float *>(ws->data), wslot, swslot, (int32_t)K, (int32_t)N,
      static_cast<uint16_t *>(out->data), glu, as_stream(stream)));
}

ep_status_t ep_expert_gemm_fp8(ep_handle_t h, const ep_tensor_t *recv_tokens,
                               const ep_tensor_t *recv_scales, const ep_tensor_t *expert_weights,
                               const ep_tensor_t *expert_scales, const ep_tensor_t *slot_weights,
                               const ep_tensor_t *slot_scales, ep_tensor_t *out, void *stream) {
  return expert_gemm_fp8(h, recv_tokens, recv_scales, expert_weights, expert_scales, slot_weights,
                         slot_scales, out, stream, false);
}

ep_status_t ep_expert_gemm_fp8_swiglu(ep_handle_t h, const ep_tensor_t *recv_tokens,
                                      const ep_tensor_t *recv_scales,
                                      const ep_tensor_t *expert_weights,
                                      const ep_tensor_t *expert_scales,
                                      const ep_tensor_t *slot_weights,
                                      const ep_tensor_t *slot_scales, ep_tensor_t *out,
                                      void *stream) {
  return expert_gemm_fp8(h, recv_tokens, recv_scales, expert_weights, expert_scales, slot_weights,
                         slot_scales, out, stream, true);
}

// Bounds of a routing rule for E experts.
static bool rule_ok(const ep_route_rule_t *r, int32_t E) {
  return r && (r->score == EP_SCORE_SOFTMAX || r->score == EP_SCORE_SIGMOID) &&
         r->num_groups >= 1 && r->num_groups <= 64 && E % r->num_groups == 0 &&
         r->kept_groups >= 1 && r->kept_groups <= r->num_groups &&
         (r->group_score == EP_GROUP_MAX || r->group_score == EP_GROUP_TOP2) &&
         (r->renormalise == 0 || r->renormalise == 1) && std::isfinite(r->scale);
}

// fp32 or bf16 logits [T, E]; *bf16 tells which.
static ep_status_t check_logits(const ep_tensor_t *t, const epk::Geometry &g, bool *bf16) {
  if (!t) return EP_ERR_INVALID_ARG;
  *bf16 = t->dtype == EP_DTYPE_BF16;
  const ep_status_t st = check_tensor(t, EP_TAG_ROUTER_LOGITS, *bf16 ? EP_DTYPE_BF16 : EP_DTYPE_FP32);
  if (st != EP_OK) return st;
  return is_2d(t, g.T, g.E) ? EP_OK : EP_ERR_BAD_SHAPE;
}

// A [d0, d1] tensor of the given tag and dtype.
static ep_status_t check_2d(const ep_tensor_t *t, int32_t tag, int32_t dtype, int64_t d0, int64_t d1) {
  const ep_status_t st = check_tensor(t, tag, dtype);
  if (st != EP_OK) return st;
  return is_2d(t, d0, d1) ? EP_OK : EP_ERR_BAD_SHAPE;
}

ep_status_t ep_route_scored(ep_handle_t h, const ep_route_rule_t *rule, const ep_tensor_t *logits,
                            const ep_tensor_t *bias, ep_tensor_t *topk_idx,
                            ep_tensor_t *topk_weights, ep_tensor_t *scores, void *stream) {
  if (!h) return EP_ERR_INVALID_ARG;
  const epk::Geometry &g = h->geo;
  if (!rule_ok(rule, g.E)) return EP_ERR_INVALID_ARG;
  bool bf16;
  ep_status_t st = check_logits(logits, g, &bf16);
  if (st != EP_OK) return st;
  if (bias) {
    st = check_tensor(bias, EP_TAG_ROUTER_BIAS, EP_DTYPE_FP32);
    if (st != EP_OK) return st;
    if (bias->ndim != 1 || bias->sizes[0] != g.E) return EP_ERR_BAD_SHAPE;
  }
  st = check_2d(topk_idx, EP_TAG_TOPK_IDX, EP_DTYPE_INT32, g.T, g.k);
  if (st != EP_OK) return st;
  st = check_2d(topk_weights, EP_TAG_TOPK_WEIGHTS, EP_DTYPE_FP32, g.T, g.k);
  if (st != EP_OK) return st;
  if (scores) {
    st = check_2d(scores, EP_TAG_ROUTER_LOGITS, EP_DTYPE_FP32, g.T, g.E);
    if (st != EP_OK) return st;
  }
  if (!epk::route_scored_fits(g)) return EP_ERR_UNSUPPORTED;
  return hip_status(epk::launch_route_scored(
      g, *rule, logits->data, bf16, bias ? static_cast<const float *>(bias->data) : nullptr,
      static_cast<int32_t *>(topk_idx->data), static_cast<float *>(topk_weights->data),
      scores ? static_cast<float *>(scores->data) : nullptr, as_stream(stream)));
}

ep_status_t ep_route_scored_bwd(ep_handle_t h, const ep_route_rule_t *rule,
                                const ep_tensor_t *logits, const ep_tensor_t *topk_idx,
                                const ep_tensor_t *grad_topk_weights,
                                const ep_tensor_t *grad_scores, ep_tensor_t *grad_logits,
                                void *stream) {
  if (!h) return EP_ERR_INVALID_ARG;
  const epk::Geometry &g = h->geo;
  if (!rule_ok(rule, g.E)) return EP_ERR_INVALID_ARG;
  bool bf16;
  ep_status_t st = check_logits(logits, g, &bf16);
  if (st != EP_OK) return st;
  st = check_2d(topk_idx, EP_TAG_TOPK_IDX, EP_DTYPE_INT32, g.T, g.k);
  if (st != EP_OK) return st;
  st = check_2d(grad_topk_weights, EP_TAG_TOPK_WEIGHTS, EP_DTYPE_FP32, g.T, g.k);
  if (st != EP_OK) return st;
  if (grad_scores) {
    st = check_2d(grad_scores, EP_TAG_ROUTER_LOGITS, EP_DTYPE_FP32, g.T, g.E);
    if (st != EP_OK) return st;
  }
  st = check_2d(grad_logits, EP_TAG_ROUTER_LOGITS, logits->dtype, g.T, g.E);
  if (st != EP_OK) return st;
  if (!epk::route_scored_fits(g)) return EP_ERR_UNSUPPORTED;
  return hip_status(epk::launch_route_scored_bwd(
      g, h->ws, *rule, logits->data, bf16, static_cast<const int32_t *>(topk_idx->data),
      static_cast<const float *>(grad_topk_weights->data),
      grad_scores ? static_cast<const float *>(grad_scores->data) : nullptr, grad_logits->data,
      as_stream(stream)));
}

// Rows of a [.., H] tensor that passed check_tensor, if the row kernels take
// it (H a multiple of 8, rows an int32); false if they do not.
static bool row_tensor(const ep_tensor_t *t, int64_t *rows, int64_t *H) {
  if (t->ndim < 2) return false;
  *H = t->sizes[t->ndim - 1];
  if (*H <= 0 || *H % 8 != 0) return false;
  *rows = numel(t) / *H;
  return *rows <= INT32_MAX;
}

// bf16 or fp32 rows of the given shape; *fp32 tells which.
static ep_status_t check_stream_rows(const ep_tensor_t *t, int64_t rows, int64_t H, bool *fp32) {
  if (!t) return EP_ERR_INVALID_ARG;
  *fp32 = t->dtype == EP_DTYPE_FP32;
  const ep_status_t st = check_tensor(t, EP_TAG_TOKENS, *fp32 ? EP_DTYPE_FP32 : EP_DTYPE_BF16);
  if (st != EP_OK) return st;
  return is_rows(t, rows, H) ? EP_OK : EP_ERR_BAD_SHAPE;
}

static ep_status_t check_norm_weight(const ep_tensor_t *t, int64_t H, bool *fp32) {
  if (!t) return EP_ERR_INVALID_ARG;
  *fp32 = t->dtype == EP_DTYPE_FP32;
  const ep_status_t st = check_tensor(t, EP_TAG_NORM_WEIGHT, *fp32 ? EP_DTYPE_FP32 : EP_DTYPE_BF16);
  if (st != EP_OK) return st;
  return t->ndim == 1 && t->sizes[0] == H ? EP_OK : EP_ERR_BAD_SHAPE;
}

static bool norm_rule_ok(const ep_norm_rule_t *r) {
  return r && std::isfinite(r->eps) && r->eps >= (double)FLT_MIN && r->reserved == 0 &&
         r->quant >= EP_QUANT_NONE && r->quant <= EP_QUANT_INT8;
}

ep_status_t ep_add_rmsnorm(const ep_norm_rule_t *rule, const ep_tensor_t *x,
                           const ep_tensor_t *residual, const ep_tensor_t *weight,
                           ep_tensor_t *residual_out, ep_tensor_t *y, ep_tensor_t *codes,
                           ep_tensor_t *scales, void *stream) {
  if (!norm_rule_ok(rule)) return EP_ERR_INVALID_ARG;
  const int32_t q = rule->quant;
  if ((residual == nullptr) != (residual_out == nullptr)) return EP_ERR_INVALID_ARG;
  if ((q != EP_QUANT_NONE) != (codes != nullptr) || (codes == nullptr) != (scales == nullptr))
    return EP_ERR_INVALID_ARG;
  if (!y && !codes) return EP_ERR_INVALID_ARG;
  ep_status_t st = check_tensor(x, EP_TAG_TOKENS, EP_DTYPE_BF16);
  if (st != EP_OK) return st;
  epk::RmsNorm n{};
  int64_t T, H;
  if (!row_tensor(x, &T, &H)) return EP_ERR_BAD_SHAPE;
  if (H > epk::kRowMaxChannels) return EP_ERR_UNSUPPORTED;
  if (residual) {
    st = check_stream_rows(residual, T, H, &n.res_fp32);
    if (st != EP_OK) return st;
    bool out_fp32;
    st = check_stream_rows(residual_out, T, H, &out_fp32);
    if (st != EP_OK) return st;
    if (out_fp32 != n.res_fp32) return EP_ERR_BAD_DTYPE;
  }
  st = check_norm_weight(weight, H, &n.w_fp32);
  if (st != EP_OK) return st;
  if (y) {
    st = check_tensor(y, EP_TAG_TOKENS, EP_DTYPE_BF16);
    if (st != EP_OK) return st;
    if (!is_rows(y, T, H)) return EP_ERR_BAD_SHAPE;
  }
  if (codes) {
    const bool i8 = q == EP_QUANT_INT8;
    if (!i8 && H % 128 != 0) return EP_ERR_UNSUPPORTED;
    st = check_tensor(codes, EP_TAG_TOKENS, i8 ? EP_DTYPE_INT8 : EP_DTYPE_FP8_E4M3);
    if (st != EP_OK) return st;
    if (!is_rows(codes, T, H)) return EP_ERR_BAD_SHAPE;
    st = check_tensor(scales, i8 ? EP_TAG_ROW_SCALES : EP_TAG_FP8_SCALES, EP_DTYPE_FP32);
    if (st != EP_OK) return st;
    if (i8 ? numel(scales) != T : !is_rows(scales, T, H / 128)) return EP_ERR_BAD_SHAPE;
  }
  n.x = x->data;
  n.residual = residual ? residual->data : nullptr;
  n.w = weight->data;
  n.hidden = residual_out ? residual_out->data : nullptr;
  n.y = y ? y->data : nullptr;
  n.codes = codes ? static_cast<uint8_t *>(codes->data) : nullptr;
  n.scales = scales ? static_cast<float *>(scales->data) : nullptr;
  n.T = (int32_t)T;
  n.H = (int32_t)H;
  n.quant = q;
  n.eps = rule->eps;
  return hip_status(epk::launch_add_rmsnorm(n, as_stream(stream)));
}

ep_status_t ep_add_rmsnorm_bwd_workspace_bytes(int64_t rows, int32_t H, size_t *bytes) {
  if (!bytes || rows < 0 || rows > INT32_MAX || H < 8 || H % 8 != 0 || H > epk::kRowMaxChannels)
    return EP_ERR_INVALID_ARG;
  *bytes = sizeof(float) * (size_t)epk::norm_bwd_groups((int32_t)rows, H) * (size_t)H;
  return EP_OK;
}

ep_status_t ep_add_rmsnorm_bwd(const ep_norm_rule_t *rule, const ep_tensor_t *hidden,
                               const ep_tensor_t *weight, const ep_tensor_t *grad_y,
                               const ep_tensor_t *grad_residual_out, ep_tensor_t *grad,
                               ep_tensor_t *grad_weight, ep_tensor_t *workspace, void *stream) {
  if (!norm_rule_ok(rule) || rule->quant != EP_QUANT_NONE || !hidden) return EP_ERR_INVALID_ARG;
  epk::RmsNormBwd n{};
  n.h_fp32 = hidden->dtype == EP_DTYPE_FP32;
  ep_status_t st = check_tensor(hidden, EP_TAG_TOKENS, n.h_fp32 ? EP_DTYPE_FP32 : EP_DTYPE_BF16);
  if (st != EP_OK) return st;
  int64_t T, H;
  if (!row_tensor(hidden, &T, &H)) return EP_ERR_BAD_SHAPE;
  if (H > epk::kRowMaxChannels) return EP_ERR_UNSUPPORTED;
  st = check_norm_weight(weight, H, &n.w_fp32);
  if (st != EP_OK) return st;
  st = check_tensor(grad_y, EP_TAG_TOKENS, EP_DTYPE_BF16);
  if (st != EP_OK) return st;
  if (!is_rows(grad_y, T, H)) return EP_ERR_BAD_SHAPE;
  bool fp32;
  if (grad_residual_out) {
    st = check_stream_rows(grad_residual_out, T, H, &fp32);
    if (st != EP_OK) return st;
    if (fp32 != n.h_fp32) return EP_ERR_BAD_DTYPE;
  }
  st = check_stream_rows(grad, T, H, &fp32);
  if (st != EP_OK) return st;
  if (fp32 != n.h_fp32) return EP_ERR_BAD_DTYPE;
  if (grad_weight) {
    st = check_tensor(grad_weight, EP_TAG_NORM_WEIGHT, EP_DTYPE_FP32);
    if (st != EP_OK) return st;
    if (grad_weight->ndim != 1 || grad_weight->sizes[0] != H) return EP_ERR_BAD_SHAPE;
    const int64_t need = (int64_t)epk::norm_bwd_groups((int32_t)T, (int32_t)H) * H;
    if (need > 0) {
      st = check_tensor(workspace, EP_TAG_WORKSPACE, EP_DTYPE_FP32);
      if (st != EP_OK) return st;
      if (workspace->ndim != 1) return EP_ERR_BAD_SHAPE;
      if (workspace->sizes[0] < need) return EP_ERR_WORKSPACE_TOO_SMALL;
      n.part = static_cast<float *>(workspace->data);
    }
    n.gw = static_cast<float *>(grad_weight->data);
  }
  n.hidden = hidden->data;
  n.w = weight->data;
  n.gy = grad_y->data;
  n.ghidden = grad_residual_out ? grad_residual_out->data : nullptr;
  n.gx = grad->data;
  n.T = (int32_t)T;
  n.H = (int32_t)H;
  n.eps = rule->eps;
  return hip_status(epk::launch_rmsnorm_bwd(n, as_stream(stream)));
}

ep_status_t ep_quantize_int8(const ep_tensor_t *tokens, ep_tensor_t *codes, ep_tensor_t *scales,
                             void *stream) {
  ep_status_t st = check_tensor(tokens, EP_TAG_TOKENS, EP_DTYPE_BF16);
  if (st != EP_OK) return st;
  st = check_tensor(codes, EP_TAG_TOKENS, EP_DTYPE_INT8);
  if (st != EP_OK) return st;
  st = check_tensor(scales, EP_TAG_ROW_SCALES, EP_DTYPE_FP32);
  if (st != EP_OK) return st;
  int64_t rows, K;
  if (!row_tensor(tokens, &rows, &K)) return EP_ERR_BAD_SHAPE;
  if (!is_rows(codes, rows, K) || numel(scales) != rows) return EP_ERR_BAD_SHAPE;
  if (K > epk::kRowMaxChannels) return EP_ERR_UNSUPPORTED;
  return hip_status(epk::launch_quantize_int8(static_cast<const uint16_t *>(tokens->data), rows,
                                              (int32_t)K, static_cast<uint8_t *>(codes->data),
                                              static_cast<float *>(scales->data),
                                              as_stream(stream)));
}

ep_status_t ep_dispatch_quantized(ep_handle_t h, const ep_tensor_t *tokens,
                                  const ep_tensor_t *token_scales,
                                  const ep_tensor_t *topk_weights, ep_tensor_t *recv_tokens,
                                  ep_tensor_t *recv_scales, ep_tensor_t *recv_topk_idx,
                                  ep_tensor_t *recv_topk_weights, void *stream) {
  if (!h || !tokens) return EP_ERR_INVALID_ARG;
  const epk::Geometry &g = h->geo;
  const int32_t H = h->g->cfg.hidden;
  const bool i8 = tokens->dtype == EP_DTYPE_INT8;
  const int32_t dt = i8 ? EP_DTYPE_INT8 : EP_DTYPE_FP8_E4M3;
  const int32_t tag = i8 ? EP_TAG_ROW_SCALES : EP_TAG_FP8_SCALES;
  ep_status_t st = check_2d(tokens, EP_TAG_TOKENS, dt, g.T, H);
  if (st != EP_OK) return st;
  if (H % (i8 ? 16 : 128) != 0) return EP_ERR_UNSUPPORTED;
  const int32_t S = i8 ? 1 : H / 128;
  const auto scales_ok = [&](const ep_tensor_t *t, int64_t rows) {
    return i8 ? numel(t) == rows : is_rows(t, rows, S);
  };
  st = check_tensor(token_scales, tag, EP_DTYPE_FP32);
  if (st != EP_OK) return st;
  if (!scales_ok(token_scales, g.T)) return EP_ERR_BAD_SHAPE;
  st = check_tensor(recv_tokens, EP_TAG_TOKENS, dt);
  if (st != EP_OK) return st;
  if (!is_rows(recv_tokens, g.rows, H)) return EP_ERR_BAD_SHAPE;
  st = check_tensor(recv_scales, tag, EP_DTYPE_FP32);
  if (st != EP_OK) return st;
  if (!scales_ok(recv_scales, g.rows)) return EP_ERR_BAD_SHAPE;
  st = check_recv_meta(g, topk_weights, recv_topk_idx, recv_topk_weights);
  if (st != EP_OK) return st;
  if (g.T >= 1 << 23) return EP_ERR_UNSUPPORTED;   // a launch counts its threads in 32 bits
  if (!h->planned) return EP_ERR_NOT_PLANNED;
  hipError_t e = epk::launch_dispatch_rows8(
      g, h->ws, static_cast<const uint8_t *>(tokens->data),
      static_cast<const float *>(token_scales->data), H, S,
      static_cast<uint8_t *>(recv_tokens->data), static_cast<float *>(recv_scales->data),
      as_stream(stream));
  if (e == hipSuccess && (recv_topk_idx || recv_topk_weights))
    e = epk::launch_recv_meta(
        g, h->ws, topk_weights ? static_cast<const float *>(topk_weights->data) : nullptr,
        recv_topk_idx ? static_cast<int32_t *>(recv_topk_idx->data) : nullptr,
        recv_topk_weights ? static_cast<float *>(recv_topk_weights->data) : nullptr,
        as_stream(stream));
  return hip_status(e);
}

static ep_status_t expert_gemm_int8(ep_handle_t h, const ep_tensor_t *recv_tokens,
                                    const ep_tensor_t *recv_scales,
                                    const ep_tensor_t *expert_weights,
                                    const ep_tensor_t *expert_scales,
                                    const ep_tensor_t *slot_weights,
                                    const ep_tensor_t *slot_scales, ep_tensor_t *out, void *stream,
                                    bool glu) {
  if (!h) return EP_ERR_INVALID_ARG;
  const epk::Geometry &g = h->geo;
  ep_status_t st = check_tensor(recv_tokens, EP_TAG_TOKENS, EP_DTYPE_INT8);
  if (st != EP_OK) return st;
  st = check_tensor(recv_scales, EP_TAG_ROW_SCALES, EP_DTYPE_FP32);
  if (st != EP_OK) return st;
  st = check_tensor(expert_weights, EP_TAG_EXPERT_WEIGHTS, EP_DTYPE_INT8);
  if (st != EP_OK) return st;
  st = check_tensor(expert_scales, EP_TAG_ROW_SCALES, EP_DTYPE_FP32);
  if (st != EP_OK) return st;
  st = check_tensor(out, EP_TAG_TOKENS, EP_DTYPE_BF16);
  if (st != EP_OK) return st;
  const ep_tensor_t *w = expert_weights;
  if (w->ndim != 3 || w->sizes[0] != g.E) return EP_ERR_BAD_SHAPE;
  const int64_t N = w->sizes[1], K = w->sizes[2];
  if (K <= 0 || K % 64 != 0 || N < 1 || N > INT32_MAX) return EP_ERR_BAD_SHAPE;
  if (glu && N % 16 != 0) return EP_ERR_BAD_SHAPE;
  if (!is_2d(expert_scales, g.E, N) || !is_rows(recv_tokens, g.rows, K) ||
      numel(recv_scales) != g.rows || !is_rows(out, g.rows, glu ? N / 2 : N))
    return EP_ERR_BAD_SHAPE;
  if ((slot_weights == nullptr) != (slot_scales == nullptr)) return EP_ERR_INVALID_ARG;
  const uint8_t *wslot = nullptr;
  const float *swslot = nullptr;
  if (slot_weights) {
    st = check_tensor(slot_weights, EP_TAG_EXPERT_WEIGHTS, EP_DTYPE_INT8);
    if (st != EP_OK) return st;
    st = check_tensor(slot_scales, EP_TAG_ROW_SCALES, EP_DTYPE_FP32);
    if (st != EP_OK) return st;
    if (g.layout != EP_LAYOUT_STATIC) return EP_ERR_UNSUPPORTED;
    const int64_t RS = (int64_t)g.R * g.S;
    const ep_tensor_t *a = slot_weights, *b = slot_scales;
    const bool w4 = a->ndim == 4 && a->sizes[0] == g.R && a->sizes[1] == g.S &&
                    a->sizes[2] == N && a->sizes[3] == K;
    const bool w3 = a->ndim == 3 && a->sizes[0] == RS && a->sizes[1] == N && a->sizes[2] == K;
    const bool s3 = b->ndim == 3 && b->sizes[0] == g.R && b->sizes[1] == g.S && b->sizes[2] == N;
    if ((!w4 && !w3) || (!s3 && !is_2d(b, RS, N))) return EP_ERR_BAD_SHAPE;
    wslot = static_cast<const uint8_t *>(a->data);
    swslot = static_cast<const float *>(b->data);
  }
  if (K > epk::kI8MaxK || !epk::gemm_int8_fits(g, (int32_t)K, (int32_t)N)) return EP_ERR_UNSUPPORTED;
  if (!h->planned) return EP_ERR_NOT_PLANNED;
  return hip_status(epk::launch_grouped_gemm_int8(
      g, h->ws, static_cast<const uint8_t *>(recv_tokens->data),
      static_cast<const float *>(recv_scales->data), static_cast<const uint8_t *>(w->data),
      static_cast<const float *>(expert_scales->data), wslot, swslot, (int32_t)K, (int32_t)N,
      static_cast<uint16_t *>(out->data), glu, as_stream(stream)));
}

ep_status_t ep_expert_gemm_int8(ep_handle_t h, const ep_tensor_t *recv_tokens,
                                const ep_tensor_t *recv_scales, const ep_tensor_t *expert_weights,
                                const ep_tensor_t *expert_scales, const ep_tensor_t *slot_weights,
                                const ep_tensor_t *slot_scales, ep_tensor_t *out, void *stream) {
  return expert_gemm_int8(h, recv_tokens, recv_scales, expert_weights, expert_scales, slot_weights,
                          slot_scales, out, stream, false);
}

ep_status_t ep_expert_gemm_int8_swiglu(ep_handle_t h, const ep_tensor_t *recv_tokens,
                                       const ep_tensor_t *recv_scales,
                                       const ep_tensor_t *expert_weights,
                                       const ep_tensor_t *expert_scales,
                                       const ep_tensor_t *slot_weights,
                                       const ep_tensor_t *slot_scales, ep_tensor_t *out,
                                       void *stream) {
  return expert_gemm_int8(h, recv_tokens, recv_scales, expert_weights, expert_scales, slot_weights,
                          slot_scales, out, stream, true);
}

// ---------------------------------------------------------------------------
// the dense half of a layer

// The generator's view and probability of a call; p 0 with no state is no dropout.
static ep_status_t check_dropout(double p, const ep_tensor_t *rng, epk::Dropout *d) {
  if (!(p >= 0.0 && p <= 1.0)) return EP_ERR_INVALID_ARG;
  const ep_status_t st = check_tensor(rng, EP_TAG_RNG_STATE, EP_DTYPE_INT32);
  if (st != EP_OK) return st;
  if (rng->ndim != 1 || rng->sizes[0] != 4) return EP_ERR_BAD_SHAPE;
  d->rng = static_cast<const int32_t *>(rng->data);
  d->threshold = (uint32_t)std::floor((1.0 - p) * 65536.0 + 0.5);
  d->scale = d->threshold ? (float)(65536.0 / d->threshold) : 0.0f;
  return EP_OK;
}

ep_status_t ep_dropout(const ep_dropout_rule_t *rule, const ep_tensor_t *rng, const ep_tensor_t *x,
                       const ep_tensor_t *residual, ep_tensor_t *out, void *stream) {
  if (!rule || !x || !out) return EP_ERR_INVALID_ARG;
  epk::DropoutAdd n{};
  ep_status_t st = check_dropout(rule->p, rng, &n.drop);
  if (st != EP_OK) return st;
  n.x_fp32 = x->dtype == EP_DTYPE_FP32;
  st = check_tensor(x, EP_TAG_TOKENS, n.x_fp32 ? EP_DTYPE_FP32 : EP_DTYPE_BF16);
  if (st != EP_OK) return st;
  int64_t T, H;
  if (!row_tensor(x, &T, &H)) return EP_ERR_BAD_SHAPE;
  st = check_stream_rows(out, T, H, &n.out_fp32);
  if (st != EP_OK) return st;
  if (residual) {
    bool fp32;
    st = check_stream_rows(residual, T, H, &fp32);
    if (st != EP_OK) return st;
    if (fp32 != n.out_fp32) return EP_ERR_BAD_DTYPE;
    n.residual = residual->data;
  }
  n.x = x->data;
  n.out = out->data;
  n.count = T * H;
  return hip_status(epk::launch_dropout(n, as_stream(stream)));
}

static bool layernorm_rule_ok(const ep_layernorm_rule_t *r) {
  return r && std::isfinite(r->eps) && r->eps >= (double)FLT_MIN && r->reserved == 0 &&
         r->dropout >= 0.0 && r->dropout <= 1.0 && r->quant >= EP_QUANT_NONE &&
         r->quant <= EP_QUANT_INT8;
}

ep_status_t ep_add_layernorm(const ep_layernorm_rule_t *rule, const ep_layernorm_t *t, void *stream) {
  if (!layernorm_rule_ok(rule) || !t) return EP_ERR_INVALID_ARG;
  const int32_t q = rule->quant;
  const bool drop = rule->dropout != 0.0;
  if (drop != (t->rng != nullptr) || (t->residual || drop) != (t->residual_out != nullptr))
    return EP_ERR_INVALID_ARG;
  if ((q != EP_QUANT_NONE) != (t->codes != nullptr) || (t->codes == nullptr) != (t->scales == nullptr))
    return EP_ERR_INVALID_ARG;
  if (!t->y && !t->codes) return EP_ERR_INVALID_ARG;
  ep_status_t st = check_tensor(t->x, EP_TAG_TOKENS, EP_DTYPE_BF16);
  if (st != EP_OK) return st;
  epk::LayerNorm n{};
  int64_t T, H;
  if (!row_tensor(t->x, &T, &H)) return EP_ERR_BAD_SHAPE;
  if (H > epk::kRowMaxChannels) return EP_ERR_UNSUPPORTED;
  if (drop) {
    st = check_dropout(rule->dropout, t->rng, &n.drop);
    if (st != EP_OK) return st;
  }
  if (t->residual) {
    st = check_stream_rows(t->residual, T, H, &n.res_fp32);
    if (st != EP_OK) return st;
  }
  if (t->residual_out) {
    bool out_fp32;
    st = check_stream_rows(t->residual_out, T, H, &out_fp32);
    if (st != EP_OK) return st;
    if (out_fp32 != n.res_fp32) return EP_ERR_BAD_DTYPE;
  }
  st = check_norm_weight(t->weight, H, &n.w_fp32);
  if (st != EP_OK) return st;
  if (t->bias) {
    bool fp32;
    st = check_norm_weight(t->bias, H, &fp32);
    if (st != EP_OK) return st;
    if (fp32 != n.w_fp32) return EP_ERR_BAD_DTYPE;
  }
  if (t->y) {
    st = check_tensor(t->y, EP_TAG_TOKENS, EP_DTYPE_BF16);
    if (st != EP_OK) return st;
    if (!is_rows(t->y, T, H)) return EP_ERR_BAD_SHAPE;
  }
  if (t->codes) {
    const bool i8 = q == EP_QUANT_INT8;
    if (!i8 && H % 128 != 0) return EP_ERR_UNSUPPORTED;
    st = check_tensor(t->codes, EP_TAG_TOKENS, i8 ? EP_DTYPE_INT8 : EP_DTYPE_FP8_E4M3);
    if (st != EP_OK) return st;
    if (!is_rows(t->codes, T, H)) return EP_ERR_BAD_SHAPE;
    st = check_tensor(t->scales, i8 ? EP_TAG_ROW_SCALES : EP_TAG_FP8_SCALES, EP_DTYPE_FP32);
    if (st != EP_OK) return st;
    if (i8 ? numel(t->scales) != T : !is_rows(t->scales, T, H / 128)) return EP_ERR_BAD_SHAPE;
  }
  n.x = t->x->data;
  n.residual = t->residual ? t->residual->data : nullptr;
  n.w = t->weight->data;
  n.b = t->bias ? t->bias->data : nullptr;
  n.hidden = t->residual_out ? t->residual_out->data : nullptr;
  n.y = t->y ? t->y->data : nullptr;
  n.codes = t->codes ? static_cast<uint8_t *>(t->codes->data) : nullptr;
  n.scales = t->scales ? static_cast<float *>(t->scales->data) : nullptr;
  n.T = (int32_t)T;
  n.H = (int32_t)H;
  n.quant = q;
  n.eps = rule->eps;
  return hip_status(epk::launch_add_layernorm(n, as_stream(stream)));
}

ep_status_t ep_add_layernorm_bwd_workspace_bytes(int64_t rows, int32_t H, size_t *bytes) {
  if (!bytes || rows < 0 || rows > INT32_MAX || H < 8 || H % 8 != 0 || H > epk::kRowMaxChannels)
    return EP_ERR_INVALID_ARG;
  // partial rows of grad_weight and of grad_bias
  *bytes = sizeof(float) * 2 * (size_t)epk::layernorm_bwd_groups((int32_t)rows, H) * (size_t)H;
  return EP_OK;
}

ep_status_t ep_add_layernorm_bwd(const ep_layernorm_rule_t *rule, const ep_layernorm_bwd_t *t,
                                 void *stream) {
  if (!layernorm_rule_ok(rule) || rule->quant != EP_QUANT_NONE || !t || !t->hidden)
    return EP_ERR_INVALID_ARG;
  const bool drop = rule->dropout != 0.0;
  if (drop != (t->rng != nullptr) || drop != (t->grad_x != nullptr) || (!drop && !t->grad))
    return EP_ERR_INVALID_ARG;
  epk::LayerNormBwd n{};
  n.h_fp32 = t->hidden->dtype == EP_DTYPE_FP32;
  ep_status_t st = check_tensor(t->hidden, EP_TAG_TOKENS, n.h_fp32 ? EP_DTYPE_FP32 : EP_DTYPE_BF16);
  if (st != EP_OK) return st;
  int64_t T, H;
  if (!row_tensor(t->hidden, &T, &H)) return EP_ERR_BAD_SHAPE;
  if (H > epk::kRowMaxChannels) return EP_ERR_UNSUPPORTED;
  if (drop) {
    st = check_dropout(rule->dropout, t->rng, &n.drop);
    if (st != EP_OK) return st;
    st = check_tensor(t->grad_x, EP_TAG_TOKENS, EP_DTYPE_BF16);
    if (st != EP_OK) return st;
    if (!is_rows(t->grad_x, T, H)) return EP_ERR_BAD_SHAPE;
    n.gx = t->grad_x->data;
  }
  st = check_norm_weight(t->weight, H, &n.w_fp32);
  if (st != EP_OK) return st;
  st = check_tensor(t->grad_y, EP_TAG_TOKENS, EP_DTYPE_BF16);
  if (st != EP_OK) return st;
  if (!is_rows(t->grad_y, T, H)) return EP_ERR_BAD_SHAPE;
  bool fp32;
  if (t->grad_residual_out) {
    st = check_stream_rows(t->grad_residual_out, T, H, &fp32);
    if (st != EP_OK) return st;
    if (fp32 != n.h_fp32) return EP_ERR_BAD_DTYPE;
    n.ghidden = t->grad_residual_out->data;
  }
  if (t->grad) {
    st = check_stream_rows(t->grad, T, H, &fp32);
    if (st != EP_OK) return st;
    if (fp32 != n.h_fp32) return EP_ERR_BAD_DTYPE;
    n.gh = t->grad->data;
  }
  for (ep_tensor_t *g : {t->grad_weight, t->grad_bias}) {
    if (!g) continue;
    st = check_tensor(g, EP_TAG_NORM_WEIGHT, EP_DTYPE_FP32);
    if (st != EP_OK) return st;
    if (g->ndim != 1 || g->sizes[0] != H) return EP_ERR_BAD_SHAPE;
  }
  if (t->grad_weight || t->grad_bias) {
    const int64_t need = (int64_t)epk::layernorm_bwd_groups((int32_t)T, (int32_t)H) * 2 * H;
    if (need > 0) {
      st = check_tensor(t->workspace, EP_TAG_WORKSPACE, EP_DTYPE_FP32);
      if (st != EP_OK) return st;
      if (t->workspace->ndim != 1) return EP_ERR_BAD_SHAPE;
      if (t->workspace->sizes[0] < need) return EP_ERR_WORKSPACE_TOO_SMALL;
      n.part = static_cast<float *>(t->workspace->data);
    }
    n.gw = t->grad_weight ? static_cast<float *>(t->grad_weight->data) : nullptr;
    n.gb = t->grad_bias ? static_cast<float *>(t->grad_bias->data) : nullptr;
  }
  n.hidden = t->hidden->data;
  n.w = t->weight->data;
  n.gy = t->grad_y->data;
  n.T = (int32_t)T;
  n.H = (int32_t)H;
  n.eps = rule->eps;
  return hip_status(epk::launch_layernorm_bwd(n, as_stream(stream)));
}

ep_status_t ep_quantize_fp8_2d(const ep_fp8_2d_rule_t *rule, const ep_tensor_t *x, ep_tensor_t *codes,
                               ep_tensor_t *scales, ep_tensor_t *codes_t, ep_tensor_t *scales_t,
                               void *stream) {
  if (!rule || (rule->fp8_scales != EP_FP8_SCALES_AMAX && rule->fp8_scales != EP_FP8_SCALES_POW2) ||
      (rule->block != EP_FP8_BLOCK_ROWS && rule->block != EP_FP8_BLOCK_SQUARE))
    return EP_ERR_INVALID_ARG;
  if ((codes == nullptr) != (scales == nullptr) || (codes_t == nullptr) != (scales_t == nullptr) ||
      (!codes && !codes_t))
    return EP_ERR_INVALID_ARG;
  ep_status_t st = check_tensor(x, EP_TAG_TOKENS, EP_DTYPE_BF16);
  if (st != EP_OK) return st;
  if (x->ndim != 2) return EP_ERR_BAD_SHAPE;
  const int64_t R = x->sizes[0], C = x->sizes[1];
  if (C <= 0 || C % 128 != 0) return EP_ERR_BAD_SHAPE;
  const int64_t rb = (R + 127) / 128, cb = C / 128;
  if (R > INT32_MAX - 127 || C > INT32_MAX - 127 || rb * cb >= (int64_t)1 << 24) return EP_ERR_UNSUPPORTED;
  const bool sq = rule->block == EP_FP8_BLOCK_SQUARE;
  if (codes) {
    st = check_tensor(codes, EP_TAG_TOKENS, EP_DTYPE_FP8_E4M3);
    if (st != EP_OK) return st;
    st = check_tensor(scales, EP_TAG_FP8_SCALES, EP_DTYPE_FP32);
    if (st != EP_OK) return st;
    if (!is_2d(codes, R, C) || !is_2d(scales, sq ? rb : R, cb)) return EP_ERR_BAD_SHAPE;
  }
  if (codes_t) {
    st = check_tensor(codes_t, EP_TAG_TOKENS, EP_DTYPE_FP8_E4M3);
    if (st != EP_OK) return st;
    st = check_tensor(scales_t, EP_TAG_FP8_SCALES, EP_DTYPE_FP32);
    if (st != EP_OK) return st;
    if (!is_2d(codes_t, C, rb * 128) || !is_2d(scales_t, sq ? cb : C, rb)) return EP_ERR_BAD_SHAPE;
  }
  epk::Quantize2d n{};
  n.x = static_cast<const uint16_t *>(x->data);
  n.R = (int32_t)R;
  n.C = (int32_t)C;
  n.codes = codes ? static_cast<uint8_t *>(codes->data) : nullptr;
  n.scales = scales ? static_cast<float *>(scales->data) : nullptr;
  n.codes_t = codes_t ? static_cast<uint8_t *>(codes_t->data) : nullptr;
  n.scales_t = scales_t ? static_cast<float *>(scales_t->data) : nullptr;
  n.square = sq;
  n.pow2 = rule->fp8_scales == EP_FP8_SCALES_POW2;
  return hip_status(epk::launch_quantize_2d(n, as_stream(stream)));
}

ep_status_t ep_linear_fp8(const ep_linear_rule_t *rule, const ep_tensor_t *x,
                          const ep_tensor_t *x_scales, const ep_tensor_t *w,
                          const ep_tensor_t *w_scales, const ep_tensor_t *addend, ep_tensor_t *out,
                          ep_tensor_t *status, void *stream) {
  if (!rule || (rule->fp8_scales != EP_FP8_SCALES_AMAX && rule->fp8_scales != EP_FP8_SCALES_POW2) ||
      (rule->swiglu != 0 && rule->swiglu != 1) || !out)
    return EP_ERR_INVALID_ARG;
  const bool glu = rule->swiglu == 1;
  if (glu && addend) return EP_ERR_INVALID_ARG;
  epk::Linear n{};
  ep_status_t st = check_tensor(x, EP_TAG_TOKENS, EP_DTYPE_FP8_E4M3);
  if (st != EP_OK) return st;
  st = check_tensor(x_scales, EP_TAG_FP8_SCALES, EP_DTYPE_FP32);
  if (st != EP_OK) return st;
  st = check_tensor(w, EP_TAG_EXPERT_WEIGHTS, EP_DTYPE_FP8_E4M3);
  if (st != EP_OK) return st;
  st = check_tensor(w_scales, EP_TAG_FP8_SCALES, EP_DTYPE_FP32);
  if (st != EP_OK) return st;
  if (x->ndim < 2 || w->ndim != 2) return EP_ERR_BAD_SHAPE;
  const int64_t K = x->sizes[x->ndim - 1], N = w->sizes[0];
  if (K % 128 != 0 || w->sizes[1] != K) return EP_ERR_BAD_SHAPE;
  int64_t M = 1;   // (K may be 0: the weight gradient of no tokens)
  for (int i = 0; i + 1 < x->ndim; ++i) M *= x->sizes[i];
  if (K > epk::kLinearMaxK || M > INT32_MAX - 255 || N > INT32_MAX - 255) return EP_ERR_UNSUPPORTED;
  if (glu && N % 16 != 0) return EP_ERR_BAD_SHAPE;
  if (!is_rows(x_scales, M, K / 128)) return EP_ERR_BAD_SHAPE;
  if (is_2d(w_scales, (N + 127) / 128, K / 128)) n.row_scales = false;   // (N = 1: the same)
  else if (is_2d(w_scales, N, K / 128)) n.row_scales = true;
  else return EP_ERR_BAD_SHAPE;
  st = check_stream_rows(out, M, glu ? N / 2 : N, &n.out_fp32);
  if (st != EP_OK) return st;
  if (glu && n.out_fp32) return EP_ERR_BAD_DTYPE;
  if (addend) {
    bool fp32;
    st = check_stream_rows(addend, M, N, &fp32);
    if (st != EP_OK) return st;
    if (fp32 != n.out_fp32) return EP_ERR_BAD_DTYPE;
    n.addend = addend->data;
  }
  if (status) {
    st = check_tensor(status, EP_TAG_STATUS, EP_DTYPE_INT32);
    if (st != EP_OK) return st;
    if (status->ndim != 1 || status->sizes[0] != 1) return EP_ERR_BAD_SHAPE;
    n.status = static_cast<uint32_t *>(status->data);
  }
  n.x = static_cast<const uint8_t *>(x->data);
  n.w = static_cast<const uint8_t *>(w->data);
  n.xs = static_cast<const float *>(x_scales->data);
  n.ws = static_cast<const float *>(w_scales->data);
  n.out = out->data;
  n.M = (int32_t)M;
  n.N = (int32_t)N;
  n.K = (int32_t)K;
  n.glu = glu;
  n.pow2 = rule->fp8_scales == EP_FP8_SCALES_POW2;
  if (!epk::linear_fp8_fits(n)) return EP_ERR_UNSUPPORTED;
  return hip_status(epk::launch_linear_fp8(n, as_stream(stream)));
}

ep_status_t ep_run_calls(const ep_call_t *calls, int32_t n, int32_t *failed) {
  if (failed != nullptr) *failed = 0;
  if (n < 0 || (n > 0 && calls == nullptr)) return EP_ERR_INVALID_ARG;
  for (int32_t i = 0; i < n; ++i) {
    const ep_call_t &c = calls[i];
    const auto h = static_cast<ep_handle_t>(c.p[0]);
    const auto t = [&c](int k) { return static_cast<ep_tensor_t *>(c.p[k]); };
    ep_status_t st;
    switch (c.op) {
      case EP_OP_ROUTE: st = ep_route(h, t(1), t(2), t(3), c.p[4]); break;
      case EP_OP_ROUTE_PLAN: st = ep_route_plan(h, t(1), t(2), t(3), c.p[4]); break;
      case EP_OP_PLAN: st = ep_plan(h, t(1), c.p[2]); break;
      case EP_OP_DISPATCH: st = ep_dispatch(h, t(1), t(2), t(3), t(4), t(5), t(6), c.p[7]); break;
      case EP_OP_PLAN_DISPATCH:
        st = ep_plan_dispatch(h, t(1), t(2), t(3), t(4), t(5), t(6), t(7), c.p[8]);
        break;
      case EP_OP_QUANTIZE_FP8: st = ep_quantize_fp8(t(0), t(1), t(2), c.i0, c.p[3]); break;
      case EP_OP_COMBINE: st = ep_combine(h, t(1), t(2), t(3), c.p[4]); break;
      case EP_OP_COMBINE_BWD: st = ep_combine_bwd(h, t(1), t(2), t(3), t(4), t(5), c.p[6]); break;
      case EP_OP_DUP_GRAD_REDUCE: st = ep_dup_grad_reduce(h, t(1), t(2), t(3), c.p[4]); break;
      case EP_OP_PREFETCH_REPLICAS: st = ep_prefetch_replicas(h, t(1), t(2), c.p[3]); break;
      case EP_OP_EXPERT_GEMM: st = ep_expert_gemm(h, t(1), t(2), t(3), t(4), c.p[5]); break;
      case EP_OP_EXPERT_GEMM_SWIGLU:
        st = ep_expert_gemm_swiglu(h, t(1), t(2), t(3), t(4), c.p[5]);
        break;
      case EP_OP_EXPERT_GEMM_FP8:
        st = ep_expert_gemm_fp8(h, t(1), t(2), t(3), t(4), t(5), t(6), t(7), c.p[8]);
        break;
      case EP_OP_EXPERT_GEMM_FP8_SWIGLU:
        st = ep_expert_gemm_fp8_swiglu(h, t(1), t(2), t(3), t(4), t(5), t(6), t(7), c.p[8]);
        break;
      case EP_OP_ROUTE_SCORED:
        st = ep_route_scored(h, static_cast<const ep_route_rule_t *>(c.p[1]), t(2), t(3), t(4), t(5),
                             t(6), c.p[7]);
        break;
      case EP_OP_ROUTE_SCORED_BWD:
        st = ep_route_scored_bwd(h, static_cast<const ep_route_rule_t *>(c.p[1]), t(2), t(3), t(4),
                                 t(5), t(6), c.p[7]);
        break;
      case EP_OP_ADD_RMSNORM:
        st = ep_add_rmsnorm(static_cast<const ep_norm_rule_t *>(c.p[0]), t(1), t(2), t(3), t(4), t(5),
                            t(6), t(7), c.p[8]);
        break;
      case EP_OP_ADD_RMSNORM_BWD:
        st = ep_add_rmsnorm_bwd(static_cast<const ep_norm_rule_t *>(c.p[0]), t(1), t(2), t(3), t(4),
                                t(5), t(6), t(7), c.p[8]);
        break;
      case EP_OP_QUANTIZE_INT8: st = ep_quantize_int8(t(0), t(1), t(2), c.p[3]); break;
      case EP_OP_DISPATCH_QUANTIZED:
        st = ep_dispatch_quantized(h, t(1), t(2), t(3), t(4), t(5), t(6), t(7), c.p[8]);
        break;
      case EP_OP_EXPERT_GEMM_INT8:
        st = ep_expert_gemm_int8(h, t(1), t(2), t(3), t(4), t(5), t(6), t(7), c.p[8]);
        break;
      case EP_OP_EXPERT_GEMM_INT8_SWIGLU:
        st = ep_expert_gemm_int8_swiglu(h, t(1), t(2), t(3), t(4), t(5), t(6), t(7), c.p[8]);
        break;
      case EP_OP_DROPOUT:
        st = ep_dropout(static_cast<const ep_dropout_rule_t *>(c.p[0]), t(1), t(2), t(3), t(4), c.p[5]);
        break;
      case EP_OP_ADD_LAYERNORM:
        st = ep_add_layernorm(static_cast<const ep_layernorm_rule_t *>(c.p[0]),
                              static_cast<const ep_layernorm_t *>(c.p[1]), c.p[2]);
        break;
      case EP_OP_ADD_LAYERNORM_BWD:
        st = ep_add_layernorm_bwd(static_cast<const ep_layernorm_rule_t *>(c.p[0]),
                                  static_cast<const ep_layernorm_bwd_t *>(c.p[1]), c.p[2]);
        break;
      case EP_OP_QUANTIZE_FP8_2D:
        st = ep_quantize_fp8_2d(static_cast<const ep_fp8_2d_rule_t *>(c.p[0]), t(1), t(2), t(3), t(4),
                                t(5), c.p[6]);
        break;
      case EP_OP_LINEAR_FP8:
        st = ep_linear_fp8(static_cast<const ep_linear_rule_t *>(c.p[0]), t(1), t(2), t(3), t(4), t(5),
                           t(6), t(7), c.p[8]);
        break;
      default: st = EP_ERR_INVALID_ARG; break;
    }
    if (st != EP_OK) {
      if (failed != nullptr) *failed = i;
      return st;
    }
  }
  if (failed != nullptr) *failed = n;
  return EP_OK;
}

}  // extern "C"
