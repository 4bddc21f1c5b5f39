"""MoE expert-parallel token dispatch / combine / static-shape planner for
MI355X (gfx950).

A thin binding over ``libep_mi355x.so`` (C ABI in ``include/ep.h``).  It only
marshals arguments: torch tensors provide device memory and the stream, and
every step of the path runs in the library's HIP kernels.  There is no CPU
or PyTorch fallback: if the library is missing the calls raise.

The functions ``ep_group_create`` ... ``ep_dup_grad_reduce`` mirror the C
entry points one to one.  ``Group`` / ``Handle`` / ``Buffer`` wrap them in
the group -> handle -> dispatch -> expert -> combine flow of the NCCL EP
paper (listing, Table II and Figure 2), and ``Buffer.dispatch`` returns
``recv_x, recv_i, recv_w, handle, event`` like that paper's Table V.
``Buffer.add_rmsnorm``, ``Handle.route_scored``, ``Buffer.dispatch_quantized``,
``Buffer.expert_gemm_int8`` and ``Buffer.quantize_int8`` are the layer's front
and its INT8 path; their arguments are marshalled in C++ (``_marshal``).
"""

from __future__ import annotations

import ctypes
import os
import threading
from ctypes import POINTER, c_int32, c_int64, c_size_t, c_uint32, c_void_p

import torch

__all__ = [
    "EpError", "LAYOUT_LL", "LAYOUT_HT", "LAYOUT_STATIC", "FLAG_INDEX_RANGE", "FLAG_CAPACITY",
    "FLAG_SLOT_BUDGET", "FLAG_PLAN_STALL", "FLAG_SCALE_FORMAT", "Group", "Handle", "Buffer", "library_path", "load_library",
    "ep_status_string", "ep_group_create", "ep_group_destroy", "ep_group_recv_rows",
    "ep_handle_workspace_bytes", "ep_handle_create", "ep_handle_create_static", "ep_handle_destroy",
    "ep_handle_query",
    "ep_handle_status", "ep_route", "ep_route_plan", "ep_plan", "ep_dispatch", "ep_plan_dispatch",
    "ep_quantize_fp8", "ep_combine", "ep_combine_bwd", "prepare", "Prepared",
    "ep_dup_grad_reduce", "ep_prefetch_replicas", "ep_expert_gemm", "ep_expert_gemm_fp8",
    "ep_expert_gemm_swiglu", "ep_expert_gemm_fp8_swiglu", "ep_run_calls", "ep_call_t",
    "SLOTS_TRAINING",
    "SLOTS_INFERENCE",
    "STORES_AUTO", "STORES_CACHED", "STORES_STREAMING", "FP8_SCALES_AMAX", "FP8_SCALES_POW2",
    "RouteRule", "ep_route_scored", "ep_route_scored_bwd", "ep_add_rmsnorm", "ep_add_rmsnorm_bwd",
    "ep_add_rmsnorm_bwd_workspace_bytes", "ep_quantize_int8", "ep_dispatch_quantized",
    "ep_expert_gemm_int8", "ep_expert_gemm_int8_swiglu",
]

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_NAME = "libep_mi355x.so"

LAYOUT_LL, LAYOUT_HT, LAYOUT_STATIC = 0, 1, 2
_LAYOUTS = {"ll": LAYOUT_LL, "ht": LAYOUT_HT, "static": LAYOUT_STATIC}
FLAG_INDEX_RANGE, FLAG_CAPACITY, FLAG_SLOT_BUDGET, FLAG_PLAN_STALL, FLAG_SCALE_FORMAT = 1, 2, 4, 8, 16
TAG_TOKENS, TAG_TOPK_IDX, TAG_TOPK_WEIGHTS, TAG_FP8_SCALES, TAG_EXPERT_GRADS = 0, 1, 2, 3, 4
TAG_ROUTER_LOGITS, TAG_EXPERT_WEIGHTS, TAG_ROW_SCALES, TAG_ROUTER_BIAS = 5, 6, 7, 8
TAG_NORM_WEIGHT, TAG_WORKSPACE = 9, 10
SLOTS_TRAINING, SLOTS_INFERENCE = 0, 1
_SLOT_MODES = {"training": SLOTS_TRAINING, "inference": SLOTS_INFERENCE}
STORES_AUTO, STORES_CACHED, STORES_STREAMING = 0, 1, 2
_STORES = {"auto": STORES_AUTO, "cached": STORES_CACHED, "streaming": STORES_STREAMING}
FP8_SCALES_AMAX, FP8_SCALES_POW2, FP8_SCALES_AMAX_POW2_WEIGHTS = 0, 1, 2
_FP8_SCALES = {"amax": FP8_SCALES_AMAX, "pow2": FP8_SCALES_POW2,
               "amax_pow2w": FP8_SCALES_AMAX_POW2_WEIGHTS}
SCORE_SOFTMAX, SCORE_SIGMOID = 0, 1
_SCORES = {"softmax": SCORE_SOFTMAX, "sigmoid": SCORE_SIGMOID}
GROUP_MAX, GROUP_TOP2 = 0, 1
_GROUP_SCORES = {"max": GROUP_MAX, "top2": GROUP_TOP2}
QUANT_NONE, QUANT_FP8, QUANT_FP8_POW2, QUANT_INT8 = 0, 1, 2, 3
_QUANTS = {"none": QUANT_NONE, "fp8": QUANT_FP8, "fp8_pow2": QUANT_FP8_POW2, "int8": QUANT_INT8}
_DTYPES = {torch.bfloat16: 0, torch.float32: 1, torch.float8_e4m3fn: 2, torch.int32: 3, torch.int8: 4}
_STATUS = ["EP_OK", "EP_ERR_INVALID_ARG", "EP_ERR_BAD_TAG", "EP_ERR_BAD_DTYPE",
           "EP_ERR_BAD_SHAPE", "EP_ERR_NOT_PLANNED", "EP_ERR_WORKSPACE_TOO_SMALL",
           "EP_ERR_UNSUPPORTED", "EP_ERR_HIP"]


class EpError(RuntimeError):
    def __init__(self, code: int, what: str):
        self.code = code
        name = _STATUS[code] if 0 <= code < len(_STATUS) else str(code)
        super().__init__(f"{what} failed: {name}")


class ep_tensor_t(ctypes.Structure):
    _fields_ = [("data", c_void_p), ("dtype", c_int32), ("tag", c_int32), ("ndim", c_int32),
                ("reserved", c_int32), ("sizes", c_int64 * 4)]


class ep_group_config_t(ctypes.Structure):
    _fields_ = [("num_experts", c_int32), ("num_ranks", c_int32), ("hidden", c_int32),
                ("top_k", c_int32), ("max_tokens", c_int32), ("layout", c_int32),
                ("capacity", c_int32), ("slots_per_rank", c_int32), ("slot_mode", c_int32),
                ("dispatch_stores", c_int32), ("passes_in_flight", c_int32),
                ("fp8_scales", c_int32), ("combine_stores", c_int32)]


class ep_call_t(ctypes.Structure):
    """One recorded call for ep_run_calls: op, integer argument, pointers."""
    _fields_ = [("op", c_int32), ("i0", c_int32), ("p", c_void_p * 9)]


_OPS = {"ep_route": 1, "ep_route_plan": 2, "ep_plan": 3, "ep_dispatch": 4, "ep_plan_dispatch": 5,
        "ep_quantize_fp8": 6, "ep_combine": 7, "ep_combine_bwd": 8, "ep_dup_grad_reduce": 9,
        "ep_prefetch_replicas": 10, "ep_expert_gemm": 11, "ep_expert_gemm_swiglu": 12,
        "ep_expert_gemm_fp8": 13, "ep_expert_gemm_fp8_swiglu": 14, "ep_route_scored": 15,
        "ep_route_scored_bwd": 16, "ep_add_rmsnorm": 17, "ep_add_rmsnorm_bwd": 18,
        "ep_quantize_int8": 19, "ep_dispatch_quantized": 20, "ep_expert_gemm_int8": 21,
        "ep_expert_gemm_int8_swiglu": 22}


class ep_route_rule_t(ctypes.Structure):
    _fields_ = [("score", c_int32), ("num_groups", c_int32), ("kept_groups", c_int32),
                ("group_score", c_int32), ("renormalise", c_int32), ("scale", ctypes.c_float)]


class ep_norm_rule_t(ctypes.Structure):
    _fields_ = [("eps", ctypes.c_double), ("quant", c_int32), ("reserved", c_int32)]


class ep_handle_view_t(ctypes.Structure):
    _fields_ = [("num_tokens", c_int32), ("top_k", c_int32), ("num_experts", c_int32),
                ("num_ranks", c_int32), ("recv_rows", c_int64), ("rank_rows", c_int32),
                ("max_segments", c_int32)] + [
        (n, c_void_p) for n in ("counts", "offsets", "dst", "recv_src", "status", "keep",
                                "native_row", "seg_first", "seg_count", "segments",
                                "n_segments", "load", "replica", "seg_slot")]


_lib = None
_marshal_call = None             # the C++ marshalling (csrc/marshal.cpp) and the addresses it calls
_entry: dict[str, int] = {}
_T = POINTER(ep_tensor_t)


def library_path() -> str:
    """The in-tree libep_mi355x.so, or the file EP_MI355X_LIB names (e.g. the
    host-sanitized build of the same sources)."""
    return os.environ.get("EP_MI355X_LIB") or os.path.join(_HERE, _LIB_NAME)


def _without_marshal(why: ImportError):
    """What stands for the marshalling module where it cannot be loaded (it is
    bound to the torch it was built with): the calls that need it say so."""
    reason = str(why)   # the exception itself would keep its frames

    def call(*_):
        raise RuntimeError(f"combine_ep_plan_amd._marshal cannot be loaded ({reason}): build it with"
                           " `python -m combine_ep_plan_amd.build` (there is no fallback path)")
    return call


def load_library():
    """Load libep_mi355x.so (raises if it has not been built) and the
    marshalling module (without it the entry points it marshals raise)."""
    global _lib, _marshal_call
    if _lib is not None:
        return _lib
    path = library_path()
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with `python -m combine_ep_plan_amd.build`"
                           " (there is no fallback path)")
    lib = ctypes.CDLL(path)
    S = c_int32
    sig = {
        "ep_status_string": (ctypes.c_char_p, [S]),
        "ep_group_create": (S, [POINTER(ep_group_config_t), POINTER(c_void_p)]),
        "ep_group_destroy": (S, [c_void_p]),
        "ep_group_recv_rows": (S, [c_void_p, c_int32, POINTER(c_int64)]),
        "ep_handle_workspace_bytes": (S, [c_void_p, c_int32, POINTER(c_size_t)]),
        "ep_handle_create": (S, [c_void_p, c_int32, c_void_p, c_size_t, POINTER(c_void_p)]),
        "ep_handle_create_static": (S, [c_void_p, c_int32, c_void_p, POINTER(c_void_p)]),
        "ep_handle_destroy": (S, [c_void_p]),
        "ep_handle_query": (S, [c_void_p, POINTER(ep_handle_view_t)]),
        "ep_handle_status": (S, [c_void_p, c_void_p, POINTER(c_uint32)]),
        "ep_route": (S, [c_void_p, _T, _T, _T, c_void_p]),
        "ep_route_plan": (S, [c_void_p, _T, _T, _T, c_void_p]),
        "ep_plan": (S, [c_void_p, _T, c_void_p]),
        "ep_dispatch": (S, [c_void_p, _T, _T, _T, _T, _T, _T, c_void_p]),
        "ep_plan_dispatch": (S, [c_void_p, _T, _T, _T, _T, _T, _T, _T, c_void_p]),
        "ep_quantize_fp8": (S, [_T, _T, _T, c_int32, c_void_p]),
        "ep_combine": (S, [c_void_p, _T, _T, _T, c_void_p]),
        "ep_combine_bwd": (S, [c_void_p, _T, _T, _T, _T, _T, c_void_p]),
        "ep_dup_grad_reduce": (S, [c_void_p, _T, _T, _T, c_void_p]),
        "ep_prefetch_replicas": (S, [c_void_p, _T, _T, c_void_p]),
        "ep_expert_gemm": (S, [c_void_p, _T, _T, _T, _T, c_void_p]),
        "ep_expert_gemm_fp8": (S, [c_void_p, _T, _T, _T, _T, _T, _T, _T, c_void_p]),
        "ep_expert_gemm_swiglu": (S, [c_void_p, _T, _T, _T, _T, c_void_p]),
        "ep_expert_gemm_fp8_swiglu": (S, [c_void_p, _T, _T, _T, _T, _T, _T, _T, c_void_p]),
        "ep_route_scored": (S, [c_void_p, POINTER(ep_route_rule_t), _T, _T, _T, _T, _T, c_void_p]),
        "ep_route_scored_bwd": (S, [c_void_p, POINTER(ep_route_rule_t), _T, _T, _T, _T, _T, c_void_p]),
        "ep_add_rmsnorm": (S, [POINTER(ep_norm_rule_t), _T, _T, _T, _T, _T, _T, _T, c_void_p]),
        "ep_add_rmsnorm_bwd_workspace_bytes": (S, [c_int64, c_int32, POINTER(c_size_t)]),
        "ep_add_rmsnorm_bwd": (S, [POINTER(ep_norm_rule_t), _T, _T, _T, _T, _T, _T, _T, c_void_p]),
        "ep_quantize_int8": (S, [_T, _T, _T, c_void_p]),
        "ep_dispatch_quantized": (S, [c_void_p, _T, _T, _T, _T, _T, _T, _T, c_void_p]),
        "ep_expert_gemm_int8": (S, [c_void_p, _T, _T, _T, _T, _T, _T, _T, c_void_p]),
        "ep_expert_gemm_int8_swiglu": (S, [c_void_p, _T, _T, _T, _T, _T, _T, _T, c_void_p]),
        "ep_run_calls": (S, [POINTER(ep_call_t), c_int32, POINTER(c_int32)]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
        _entry[name] = ctypes.cast(fn, c_void_p).value
    try:
        from . import _marshal
        _marshal_call = _marshal.call
    except ImportError as e:
        _marshal_call = _without_marshal(e)
    _lib = lib
    return lib


def _check(code: int, what: str) -> None:
    if code != 0:
        raise EpError(code, what)


_VIEWS: dict = {}
_VIEWS_MAX = 4096
_RECORDING = threading.local()   # prepare(): the calls being recorded and what they use
_recorders = 0                   # threads inside prepare(): the thread-local is only asked if any
_recorders_lock = threading.Lock()


def _tensor(t: torch.Tensor | None, tag: int, dev: int | None = None):
    """ep_tensor_t view of a contiguous device tensor (None -> NULL).  A view
    is a pure function of (address, dtype, shape, tag) and the library never
    writes to it, so built views are kept and reused: the marshalling of a
    call that repeats its tensors costs a dictionary lookup.  With ``dev``
    the tensor must live on that device."""
    if t is None:
        return None
    if _recorders:
        keep = getattr(_RECORDING, "keep", None)
        if keep is not None:   # a prepared call holds on to its tensors
            keep.append(t)
    on = t.get_device()
    if on < 0:
        raise ValueError("tensors passed to the library must be on the GPU")
    if dev is not None and on != dev:
        raise ValueError(f"tensor on cuda:{on}, the call runs on cuda:{dev}")
    if not t.is_contiguous():
        raise ValueError("tensors passed to the library must be contiguous")
    key = (t.data_ptr(), t.dtype, t.shape, tag)
    v = _VIEWS.get(key)
    if v is not None:
        return v
    if t.dtype not in _DTYPES:
        raise TypeError(f"unsupported dtype {t.dtype}")
    if t.dim() < 1 or t.dim() > 4:
        raise ValueError("tensors must have 1..4 dimensions")
    sizes = (c_int64 * 4)(*(int(x) for x in t.shape))
    v = ctypes.pointer(ep_tensor_t(t.data_ptr() if t.numel() > 0 else None, _DTYPES[t.dtype], tag,
                                   t.dim(), 0, sizes))
    if len(_VIEWS) >= _VIEWS_MAX:
        _VIEWS.clear()
    _VIEWS[key] = v
    return v


def _stream(stream):
    """The hipStream_t of a call: the given stream's, or the current one's."""
    if stream is None and not _recorders:   # the raw handle, without a Stream object around it
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    if stream is None:
        stream = torch.cuda.current_stream()
    keep = getattr(_RECORDING, "keep", None)
    if keep is not None:
        keep.append(stream)
    if isinstance(stream, torch.cuda.Stream):
        return c_void_p(stream.cuda_stream)
    return c_void_p(int(stream))


def _stream_object(stream) -> torch.cuda.Stream | None:
    """The Stream of a call's stream argument: None, a Stream or an address."""
    if stream is None or isinstance(stream, torch.cuda.Stream):
        return stream
    return torch.cuda.ExternalStream(int(stream))


def _event_on(stream) -> torch.cuda.Event:
    """An event behind what a call has enqueued."""
    ev = torch.cuda.Event()
    ev.record(_stream_object(stream) or torch.cuda.current_stream())
    return ev


def _hold(obj) -> None:
    """A prepared call holds on to what it points to."""
    keep = getattr(_RECORDING, "keep", None)
    if keep is not None:
        keep.append(obj)


# Compute entry points only enqueue work, so a call is fully described by the
# C function and its marshalled arguments.  prepare() records them once; its
# result makes the same C calls again without marshalling anything in Python
# (each call still validates its arguments in the library and enqueues its
# kernels).  For launch-bound loops such as low-latency decode, where the
# marshalling costs about as much host time as the launch itself.


def _enqueue(name: str, *args) -> None:
    fn = getattr(_lib or load_library(), name)
    if _recorders:
        calls = getattr(_RECORDING, "calls", None)
        if calls is not None:
            calls.append((fn, args, name))
            return
    code = fn(*args)
    if code:
        raise EpError(code, name)


class Prepared:
    """Library calls with their arguments marshalled once (see prepare),
    replayed by one ep_run_calls call.  It holds references to the tensors,
    views and streams the calls name; the tensors' storage must not be moved
    (no resize or reallocation) while it is in use."""

    def __init__(self, calls, keep):
        self.calls = tuple(calls)
        self.names = tuple(n for _, _, n in self.calls)
        self._keep = tuple(keep)
        n = len(self.calls)
        self._arr = (ep_call_t * max(n, 1))()
        for k, (_, args, name) in enumerate(self.calls):
            c = self._arr[k]
            c.op = _OPS[name]
            m = 0
            for a in args:
                if isinstance(a, c_int32):   # ep_quantize_fp8's scale format
                    c.i0 = a.value
                    continue
                # handles may come as plain addresses
                c.p[m] = a if a is None or isinstance(a, int) else ctypes.cast(a, c_void_p).value
                m += 1
        self._n = c_int32(n)
        self._failed = c_int32(0)
        self._run = load_library().ep_run_calls

    def __call__(self) -> None:
        code = self._run(self._arr, self._n, ctypes.byref(self._failed))
        if code != 0:
            raise EpError(code, self.names[self._failed.value] if self._failed.value < len(self.names)
                          else "ep_run_calls")


def prepare(fn) -> Prepared:
    """Runs ``fn()`` -- a function making compute calls of this module (route,
    plan, dispatch, combine, GEMMs, ...) -- with nothing enqueued, recording
    each C call and its marshalled arguments, and returns a Prepared object
    that repeats them.  Object-creating and querying calls are not recorded
    and must not be made inside ``fn``."""
    if getattr(_RECORDING, "calls", None) is not None:
        raise RuntimeError("prepare() does not nest")
    global _recorders
    _RECORDING.calls, _RECORDING.keep = [], []
    with _recorders_lock:
        _recorders += 1
    try:
        fn()
        return Prepared(_RECORDING.calls, _RECORDING.keep)
    finally:
        with _recorders_lock:
            _recorders -= 1
        _RECORDING.calls = _RECORDING.keep = None


# ---------------------------------------------------------------------------
# one-to-one wrappers of the C entry points
# ---------------------------------------------------------------------------

def ep_run_calls(calls, n: int) -> int:
    """Makes n recorded calls (a ctypes array of ep_call_t) in one entry into
    the library; raises at the first that fails and returns n otherwise."""
    failed = c_int32(0)
    code = load_library().ep_run_calls(calls, int(n), ctypes.byref(failed))
    if code != 0:
        raise EpError(code, f"ep_run_calls (call {failed.value})")
    return failed.value


def ep_status_string(code: int) -> str:
    return load_library().ep_status_string(int(code)).decode()


def ep_group_create(cfg: ep_group_config_t) -> int:
    out = c_void_p()
    _check(load_library().ep_group_create(ctypes.byref(cfg), ctypes.byref(out)), "ep_group_create")
    return out.value


def ep_group_destroy(g: int) -> None:
    _check(load_library().ep_group_destroy(c_void_p(g)), "ep_group_destroy")


def ep_group_recv_rows(g: int, num_tokens: int) -> int:
    out = c_int64()
    _check(load_library().ep_group_recv_rows(c_void_p(g), num_tokens, ctypes.byref(out)),
           "ep_group_recv_rows")
    return out.value


def ep_handle_workspace_bytes(g: int, num_tokens: int) -> int:
    out = c_size_t()
    _check(load_library().ep_handle_workspace_bytes(c_void_p(g), num_tokens, ctypes.byref(out)),
           "ep_handle_workspace_bytes")
    return out.value


def ep_handle_create(g: int, num_tokens: int, workspace_ptr: int, workspace_bytes: int) -> int:
    out = c_void_p()
    _check(load_library().ep_handle_create(c_void_p(g), num_tokens, c_void_p(workspace_ptr),
                                           workspace_bytes, ctypes.byref(out)), "ep_handle_create")
    return out.value


def ep_handle_create_static(g: int, num_tokens: int, stream=None) -> int:
    out = c_void_p()
    _check(load_library().ep_handle_create_static(c_void_p(g), num_tokens, _stream(stream),
                                                  ctypes.byref(out)), "ep_handle_create_static")
    return out.value


def ep_handle_destroy(h: int) -> None:
    _check(load_library().ep_handle_destroy(c_void_p(h)), "ep_handle_destroy")


def ep_handle_query(h: int) -> ep_handle_view_t:
    v = ep_handle_view_t()
    _check(load_library().ep_handle_query(c_void_p(h), ctypes.byref(v)), "ep_handle_query")
    return v


def ep_handle_status(h: int, stream=None) -> int:
    out = c_uint32()
    _check(load_library().ep_handle_status(c_void_p(h), _stream(stream), ctypes.byref(out)),
           "ep_handle_status")
    return out.value


def ep_route(h: int, logits: torch.Tensor, topk_idx: torch.Tensor,
             topk_weights: torch.Tensor, stream=None) -> None:
    _enqueue("ep_route", c_void_p(h), _tensor(logits, TAG_ROUTER_LOGITS),
             _tensor(topk_idx, TAG_TOPK_IDX), _tensor(topk_weights, TAG_TOPK_WEIGHTS),
             _stream(stream))


def ep_route_plan(h: int, logits: torch.Tensor, topk_idx: torch.Tensor,
                  topk_weights: torch.Tensor, stream=None) -> None:
    _enqueue("ep_route_plan", c_void_p(h), _tensor(logits, TAG_ROUTER_LOGITS),
             _tensor(topk_idx, TAG_TOPK_IDX), _tensor(topk_weights, TAG_TOPK_WEIGHTS),
             _stream(stream))


def ep_plan(h: int, topk_idx: torch.Tensor, stream=None) -> None:
    _enqueue("ep_plan", c_void_p(h), _tensor(topk_idx, TAG_TOPK_IDX), _stream(stream))


def ep_dispatch(h: int, tokens: torch.Tensor, topk_weights: torch.Tensor | None,
                recv_tokens: torch.Tensor, recv_scales: torch.Tensor | None = None,
                recv_topk_idx: torch.Tensor | None = None,
                recv_topk_weights: torch.Tensor | None = None, stream=None) -> None:
    _enqueue("ep_dispatch", c_void_p(h), _tensor(tokens, TAG_TOKENS),
             _tensor(topk_weights, TAG_TOPK_WEIGHTS), _tensor(recv_tokens, TAG_TOKENS),
             _tensor(recv_scales, TAG_FP8_SCALES), _tensor(recv_topk_idx, TAG_TOPK_IDX),
             _tensor(recv_topk_weights, TAG_TOPK_WEIGHTS), _stream(stream))


def ep_plan_dispatch(h: int, topk_idx: torch.Tensor, tokens: torch.Tensor,
                     topk_weights: torch.Tensor | None, recv_tokens: torch.Tensor,
                     recv_scales: torch.Tensor | None = None, recv_topk_idx: torch.Tensor | None = None,
                     recv_topk_weights: torch.Tensor | None = None, stream=None) -> None:
    _enqueue("ep_plan_dispatch", c_void_p(h), _tensor(topk_idx, TAG_TOPK_IDX),
             _tensor(tokens, TAG_TOKENS), _tensor(topk_weights, TAG_TOPK_WEIGHTS),
             _tensor(recv_tokens, TAG_TOKENS), _tensor(recv_scales, TAG_FP8_SCALES),
             _tensor(recv_topk_idx, TAG_TOPK_IDX), _tensor(recv_topk_weights, TAG_TOPK_WEIGHTS),
             _stream(stream))


def ep_quantize_fp8(tokens: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor, stream=None,
                    pow2: bool = False) -> None:
    _enqueue("ep_quantize_fp8", _tensor(tokens, TAG_TOKENS), _tensor(codes, TAG_TOKENS),
             _tensor(scales, TAG_FP8_SCALES), c_int32(FP8_SCALES_POW2 if pow2 else FP8_SCALES_AMAX),
             _stream(stream))


def ep_combine(h: int, expert_out: torch.Tensor, topk_weights: torch.Tensor | None,
               out_tokens: torch.Tensor, stream=None) -> None:
    _enqueue("ep_combine", c_void_p(h), _tensor(expert_out, TAG_TOKENS),
             _tensor(topk_weights, TAG_TOPK_WEIGHTS), _tensor(out_tokens, TAG_TOKENS),
             _stream(stream))


def ep_combine_bwd(h: int, grad_tokens: torch.Tensor, expert_out: torch.Tensor,
                   topk_weights: torch.Tensor, grad_expert_out: torch.Tensor,
                   grad_topk_weights: torch.Tensor, stream=None) -> None:
    _enqueue("ep_combine_bwd", c_void_p(h), _tensor(grad_tokens, TAG_TOKENS),
             _tensor(expert_out, TAG_TOKENS), _tensor(topk_weights, TAG_TOPK_WEIGHTS),
             _tensor(grad_expert_out, TAG_TOKENS), _tensor(grad_topk_weights, TAG_TOPK_WEIGHTS),
             _stream(stream))


def ep_dup_grad_reduce(h: int, replica_grads: torch.Tensor, replica_expert: torch.Tensor | None,
                       owner_grads: torch.Tensor, stream=None) -> None:
    _enqueue("ep_dup_grad_reduce", c_void_p(h), _tensor(replica_grads, TAG_EXPERT_GRADS),
             _tensor(replica_expert, TAG_TOPK_IDX), _tensor(owner_grads, TAG_EXPERT_GRADS),
             _stream(stream))


def ep_prefetch_replicas(h: int, expert_weights: torch.Tensor, slot_weights: torch.Tensor,
                         stream=None, scales: bool | str = False) -> None:
    """``scales``: the tensors are the fp32 scales of FP8 weights (tag
    FP8_SCALES), or with ``"row"`` those of INT8 weights (tag ROW_SCALES)."""
    tag = TAG_ROW_SCALES if scales == "row" else TAG_FP8_SCALES if scales else TAG_EXPERT_WEIGHTS
    _enqueue("ep_prefetch_replicas", c_void_p(h), _tensor(expert_weights, tag),
             _tensor(slot_weights, tag), _stream(stream))


def ep_expert_gemm(h: int, recv_tokens: torch.Tensor, expert_weights: torch.Tensor,
                   slot_weights: torch.Tensor | None, out: torch.Tensor, stream=None,
                   swiglu: bool = False) -> None:
    name = "ep_expert_gemm_swiglu" if swiglu else "ep_expert_gemm"
    _enqueue(name, c_void_p(h), _tensor(recv_tokens, TAG_TOKENS),
             _tensor(expert_weights, TAG_EXPERT_WEIGHTS),
             _tensor(slot_weights, TAG_EXPERT_WEIGHTS), _tensor(out, TAG_TOKENS), _stream(stream))


def ep_expert_gemm_swiglu(h: int, recv_tokens: torch.Tensor, expert_weights: torch.Tensor,
                          slot_weights: torch.Tensor | None, out: torch.Tensor, stream=None) -> None:
    ep_expert_gemm(h, recv_tokens, expert_weights, slot_weights, out, stream, swiglu=True)


def ep_expert_gemm_fp8(h: int, recv_tokens: torch.Tensor, recv_scales: torch.Tensor,
                       expert_weights: torch.Tensor, expert_scales: torch.Tensor,
                       slot_weights: torch.Tensor | None, slot_scales: torch.Tensor | None,
                       out: torch.Tensor, stream=None, swiglu: bool = False) -> None:
    name = "ep_expert_gemm_fp8_swiglu" if swiglu else "ep_expert_gemm_fp8"
    _enqueue(name, c_void_p(h), _tensor(recv_tokens, TAG_TOKENS),
             _tensor(recv_scales, TAG_FP8_SCALES), _tensor(expert_weights, TAG_EXPERT_WEIGHTS),
             _tensor(expert_scales, TAG_FP8_SCALES), _tensor(slot_weights, TAG_EXPERT_WEIGHTS),
             _tensor(slot_scales, TAG_FP8_SCALES), _tensor(out, TAG_TOKENS), _stream(stream))


def ep_expert_gemm_fp8_swiglu(h: int, recv_tokens: torch.Tensor, recv_scales: torch.Tensor,
                              expert_weights: torch.Tensor, expert_scales: torch.Tensor,
                              slot_weights: torch.Tensor | None, slot_scales: torch.Tensor | None,
                              out: torch.Tensor, stream=None) -> None:
    ep_expert_gemm_fp8(h, recv_tokens, recv_scales, expert_weights, expert_scales, slot_weights,
                       slot_scales, out, stream, swiglu=True)


class RouteRule:
    """How a token chooses its experts (ep_route_rule_t): ``score`` "softmax"
    or "sigmoid"; of ``num_groups`` expert groups the ``kept_groups`` best
    stay, a group counting its best expert ("max") or the sum of its two best
    ("top2"); the weights are ``scale`` times the scores, ``renormalise``d to
    sum to it or not."""

    def __init__(self, score: str | int = "softmax", num_groups: int = 1, kept_groups: int = 1,
                 group_score: str | int = "max", renormalise: bool = True, scale: float = 1.0):
        self.c = ep_route_rule_t(
            _SCORES[score] if isinstance(score, str) else int(score), num_groups, kept_groups,
            _GROUP_SCORES[group_score] if isinstance(group_score, str) else int(group_score),
            int(renormalise), scale)
        self.ptr = ctypes.pointer(self.c)
        self.addr = ctypes.addressof(self.c)


_NORM_RULES: dict = {}


def _norm_rule(eps: float, quant: str | int) -> int:
    """Address of the ep_norm_rule_t of these values (kept for the process's
    life; threads that meet the values together get the same one)."""
    r = _NORM_RULES.get((eps, quant))
    if r is None:
        q = _QUANTS[quant] if isinstance(quant, str) else int(quant)
        r = _NORM_RULES.setdefault((eps, quant), ep_norm_rule_t(eps, q, 0))
    return ctypes.addressof(r)


# Entry points that take pointers only are marshalled in C++ (csrc/marshal.cpp):
# one byte per argument, a tensor's tag or 0xFF for an address.  Recorded calls
# are described with the ctypes views above, which outlive the call.
_ADDR = 0xFF


def _call(name: str, tags: bytes, stream, *args) -> None:
    if _marshal_call is None:
        load_library()
    if _recorders and getattr(_RECORDING, "calls", None) is not None:
        dev = stream.device_index if isinstance(stream, torch.cuda.Stream) else torch.cuda.current_device()
        _enqueue(name, *(a if tag == _ADDR else _tensor(a, tag, dev) for a, tag in zip(args, tags)),
                 _stream(stream))
        return
    if stream is not None:
        stream = ((stream.device_index, stream.cuda_stream) if isinstance(stream, torch.cuda.Stream)
                  else (torch.cuda.current_device(), int(stream)))
    code = _marshal_call(_entry[name], tags, stream, *args)
    if code:
        raise EpError(code, name)


_TAGS_ROUTE = bytes((_ADDR, _ADDR, TAG_ROUTER_LOGITS, TAG_ROUTER_BIAS, TAG_TOPK_IDX, TAG_TOPK_WEIGHTS,
                     TAG_ROUTER_LOGITS))
_TAGS_ROUTE_BWD = bytes((_ADDR, _ADDR, TAG_ROUTER_LOGITS, TAG_TOPK_IDX, TAG_TOPK_WEIGHTS,
                         TAG_ROUTER_LOGITS, TAG_ROUTER_LOGITS))
_TAGS_NORM_BWD = bytes((_ADDR, TAG_TOKENS, TAG_NORM_WEIGHT, TAG_TOKENS, TAG_TOKENS, TAG_TOKENS,
                        TAG_NORM_WEIGHT, TAG_WORKSPACE))
_TAGS_QUANTIZE = bytes((TAG_TOKENS, TAG_TOKENS, TAG_ROW_SCALES))
_TAGS_GEMM_INT8 = bytes((_ADDR, TAG_TOKENS, TAG_ROW_SCALES, TAG_EXPERT_WEIGHTS, TAG_ROW_SCALES,
                         TAG_EXPERT_WEIGHTS, TAG_ROW_SCALES, TAG_TOKENS))
# with the scales of INT8 (True) or FP8 rows
_TAGS_NORM = {i8: bytes((_ADDR, TAG_TOKENS, TAG_TOKENS, TAG_NORM_WEIGHT, TAG_TOKENS, TAG_TOKENS,
                         TAG_TOKENS, TAG_ROW_SCALES if i8 else TAG_FP8_SCALES)) for i8 in (True, False)}
_TAGS_DISPATCH = {i8: bytes((_ADDR, TAG_TOKENS, t, TAG_TOPK_WEIGHTS, TAG_TOKENS, t, TAG_TOPK_IDX,
                             TAG_TOPK_WEIGHTS))
                  for i8, t in ((True, TAG_ROW_SCALES), (False, TAG_FP8_SCALES))}


def ep_route_scored(h: int, rule: RouteRule, logits: torch.Tensor, bias: torch.Tensor | None,
                    topk_idx: torch.Tensor, topk_weights: torch.Tensor,
                    scores: torch.Tensor | None = None, stream=None) -> None:
    _call("ep_route_scored", _TAGS_ROUTE, stream, h, rule.addr, logits, bias, topk_idx, topk_weights,
          scores)
    if _recorders:
        _hold(rule)


def ep_route_scored_bwd(h: int, rule: RouteRule, logits: torch.Tensor, topk_idx: torch.Tensor,
                        grad_topk_weights: torch.Tensor, grad_scores: torch.Tensor | None,
                        grad_logits: torch.Tensor, stream=None) -> None:
    _call("ep_route_scored_bwd", _TAGS_ROUTE_BWD, stream, h, rule.addr, logits, topk_idx,
          grad_topk_weights, grad_scores, grad_logits)
    if _recorders:
        _hold(rule)


def ep_add_rmsnorm(x: torch.Tensor, residual: torch.Tensor | None, weight: torch.Tensor,
                   residual_out: torch.Tensor | None, y: torch.Tensor | None,
                   codes: torch.Tensor | None = None, scales: torch.Tensor | None = None,
                   eps: float = 1e-6, quant: str | int = "none", stream=None) -> None:
    i8 = codes is not None and codes.dtype == torch.int8
    _call("ep_add_rmsnorm", _TAGS_NORM[i8], stream, _norm_rule(eps, quant), x, residual, weight,
          residual_out, y, codes, scales)


def ep_add_rmsnorm_bwd_workspace_bytes(rows: int, hidden: int) -> int:
    out = c_size_t()
    _check(load_library().ep_add_rmsnorm_bwd_workspace_bytes(rows, hidden, ctypes.byref(out)),
           "ep_add_rmsnorm_bwd_workspace_bytes")
    return out.value


def ep_add_rmsnorm_bwd(hidden: torch.Tensor, weight: torch.Tensor, grad_y: torch.Tensor,
                       grad_residual_out: torch.Tensor | None, grad: torch.Tensor,
                       grad_weight: torch.Tensor | None, workspace: torch.Tensor | None,
                       eps: float = 1e-6, stream=None) -> None:
    _call("ep_add_rmsnorm_bwd", _TAGS_NORM_BWD, stream, _norm_rule(eps, QUANT_NONE), hidden, weight,
          grad_y, grad_residual_out, grad, grad_weight, workspace)


def ep_quantize_int8(tokens: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor,
                     stream=None) -> None:
    _call("ep_quantize_int8", _TAGS_QUANTIZE, stream, tokens, codes, scales)


def ep_dispatch_quantized(h: int, tokens: torch.Tensor, token_scales: torch.Tensor,
                          topk_weights: torch.Tensor | None, recv_tokens: torch.Tensor,
                          recv_scales: torch.Tensor, recv_topk_idx: torch.Tensor | None = None,
                          recv_topk_weights: torch.Tensor | None = None, stream=None) -> None:
    _call("ep_dispatch_quantized", _TAGS_DISPATCH[tokens.dtype == torch.int8], stream, h, tokens,
          token_scales, topk_weights, recv_tokens, recv_scales, recv_topk_idx, recv_topk_weights)


def ep_expert_gemm_int8(h: int, recv_tokens: torch.Tensor, recv_scales: torch.Tensor,
                        expert_weights: torch.Tensor, expert_scales: torch.Tensor,
                        slot_weights: torch.Tensor | None, slot_scales: torch.Tensor | None,
                        out: torch.Tensor, stream=None, swiglu: bool = False) -> None:
    _call("ep_expert_gemm_int8_swiglu" if swiglu else "ep_expert_gemm_int8", _TAGS_GEMM_INT8, stream,
          h, recv_tokens, recv_scales, expert_weights, expert_scales, slot_weights, slot_scales, out)


def ep_expert_gemm_int8_swiglu(h: int, recv_tokens: torch.Tensor, recv_scales: torch.Tensor,
                               expert_weights: torch.Tensor, expert_scales: torch.Tensor,
                               slot_weights: torch.Tensor | None, slot_scales: torch.Tensor | None,
                               out: torch.Tensor, stream=None) -> None:
    ep_expert_gemm_int8(h, recv_tokens, recv_scales, expert_weights, expert_scales, slot_weights,
                        slot_scales, out, stream, swiglu=True)


# ---------------------------------------------------------------------------
# group / handle / buffer objects
# ---------------------------------------------------------------------------

class Group:
    """Long-lived configuration (experts, ranks, hidden size, top-k, layout)."""

    def __init__(self, num_experts: int, num_ranks: int, hidden: int, top_k: int,
                 max_tokens: int, layout: str | int = "ht", capacity: int = 0,
                 slots_per_rank: int = 0, slot_mode: str | int = "training",
                 dispatch_stores: str | int = "auto", passes_in_flight: int = 1,
                 fp8_scales: str | int = "amax", combine_stores: str | int = "auto"):
        self.layout = _LAYOUTS[layout] if isinstance(layout, str) else int(layout)
        mode = _SLOT_MODES[slot_mode] if isinstance(slot_mode, str) else int(slot_mode)
        stores = _STORES[dispatch_stores] if isinstance(dispatch_stores, str) else int(dispatch_stores)
        f8 = _FP8_SCALES[fp8_scales] if isinstance(fp8_scales, str) else int(fp8_scales)
        cstores = _STORES[combine_stores] if isinstance(combine_stores, str) else int(combine_stores)
        self.cfg = ep_group_config_t(num_experts, num_ranks, hidden, top_k, max_tokens,
                                     self.layout, capacity, slots_per_rank, mode, stores,
                                     passes_in_flight, f8, cstores)
        self.ptr = ep_group_create(self.cfg)

    @property
    def num_experts(self):
        return self.cfg.num_experts

    @property
    def hidden(self):
        return self.cfg.hidden

    @property
    def top_k(self):
        return self.cfg.top_k

    def recv_rows(self, num_tokens: int) -> int:
        return ep_group_recv_rows(self.ptr, num_tokens)

    def recv_shape(self, num_tokens: int) -> tuple[int, ...]:
        c = self.cfg
        rows = self.recv_rows(num_tokens)
        if self.layout == LAYOUT_LL:
            return (c.num_experts, c.capacity, c.hidden)
        if self.layout == LAYOUT_STATIC:
            return (c.num_ranks, rows // c.num_ranks, c.hidden)
        return (rows, c.hidden)

    def workspace_bytes(self, num_tokens: int) -> int:
        return ep_handle_workspace_bytes(self.ptr, num_tokens)

    def __del__(self):
        if getattr(self, "ptr", None) and _lib is not None:
            _lib.ep_group_destroy(c_void_p(self.ptr))
            self.ptr = None


class Handle:
    """Per-pass routing state over a device workspace owned by this object."""

    def __init__(self, group: Group, num_tokens: int, device: torch.device | str | None = None):
        self.group = group
        self.num_tokens = num_tokens
        nbytes = group.workspace_bytes(num_tokens)
        dev = torch.device(device) if device is not None else torch.device("cuda", torch.cuda.current_device())
        self.workspace = torch.zeros(nbytes, dtype=torch.uint8, device=dev)
        self.ptr = ep_handle_create(group.ptr, num_tokens, self.workspace.data_ptr(), nbytes)
        self._view = ep_handle_query(self.ptr)

    def route(self, logits: torch.Tensor, stream=None):
        """Top-k routing of this pass: returns (topk_idx int32 [T,k], weights fp32 [T,k])."""
        k = self.group.top_k
        idx = torch.empty((self.num_tokens, k), dtype=torch.int32, device=logits.device)
        w = torch.empty((self.num_tokens, k), dtype=torch.float32, device=logits.device)
        ep_route(self.ptr, logits, idx, w, stream)
        return idx, w

    def route_plan(self, logits: torch.Tensor, stream=None):
        """Routing and the layout of its ids in one pass (ep_route + ep_plan,
        one launch fewer): returns (topk_idx, weights); the handle is planned."""
        k = self.group.top_k
        idx = torch.empty((self.num_tokens, k), dtype=torch.int32, device=logits.device)
        w = torch.empty((self.num_tokens, k), dtype=torch.float32, device=logits.device)
        ep_route_plan(self.ptr, logits, idx, w, stream)
        return idx, w

    def route_scored(self, logits: torch.Tensor, rule: RouteRule, bias: torch.Tensor | None = None,
                     scores: bool = False, stream=None):
        """Top-k routing by scores (fp32 or bf16 logits): returns (topk_idx,
        weights), and with ``scores`` also the fp32 scores [T, E]."""
        k = self.group.top_k
        idx = torch.empty((self.num_tokens, k), dtype=torch.int32, device=logits.device)
        w = torch.empty((self.num_tokens, k), dtype=torch.float32, device=logits.device)
        s = torch.empty(logits.shape, dtype=torch.float32, device=logits.device) if scores else None
        ep_route_scored(self.ptr, rule, logits, bias, idx, w, s, stream)
        return (idx, w, s) if scores else (idx, w)

    def route_scored_bwd(self, logits: torch.Tensor, rule: RouteRule, topk_idx: torch.Tensor,
                         grad_weights: torch.Tensor, grad_scores: torch.Tensor | None = None,
                         stream=None) -> torch.Tensor:
        """Gradient of the logits from those of the weights (and scores)."""
        grad = torch.empty_like(logits)
        ep_route_scored_bwd(self.ptr, rule, logits, topk_idx, grad_weights, grad_scores, grad, stream)
        return grad

    def plan(self, topk_idx: torch.Tensor, stream=None) -> "Handle":
        ep_plan(self.ptr, topk_idx, stream)
        return self

    def status(self, stream=None) -> int:
        return ep_handle_status(self.ptr, stream)

    @property
    def recv_rows(self) -> int:
        return self._view.recv_rows

    @property
    def rank_rows(self) -> int:
        return self._view.rank_rows

    def _ws(self, ptr: int | None, count: int) -> torch.Tensor | None:
        if not ptr:
            return None
        off = ptr - self.workspace.data_ptr()
        return self.workspace[off: off + 4 * count].view(torch.int32)

    def tables(self) -> dict[str, torch.Tensor]:
        """Views (no copies) of the layout and plan tables in the workspace."""
        v = self._view
        E, R, T, k = v.num_experts, v.num_ranks, v.num_tokens, v.top_k
        out = {
            "counts": self._ws(v.counts, E),
            "offsets": self._ws(v.offsets, E + 1),
            "dst": self._ws(v.dst, T * k).view(T, k) if T * k else self._ws(v.dst, 0),
            "recv_src": self._ws(v.recv_src, v.recv_rows),
            "status": self._ws(v.status, 1),
        }
        if v.keep:
            S = self.group.cfg.slots_per_rank
            out.update({
                "keep": self._ws(v.keep, E), "native_row": self._ws(v.native_row, E),
                "seg_first": self._ws(v.seg_first, E), "seg_count": self._ws(v.seg_count, E),
                "segments": self._ws(v.segments, 5 * v.max_segments).view(v.max_segments, 5),
                "n_segments": self._ws(v.n_segments, 1), "load": self._ws(v.load, R),
                "replica": self._ws(v.replica, R * S).view(R, S),
                "seg_slot": self._ws(v.seg_slot, v.max_segments),
            })
        return out

    def __del__(self):
        if getattr(self, "ptr", None) and _lib is not None:
            _lib.ep_handle_destroy(c_void_p(self.ptr))
            self.ptr = None


class Buffer:
    """Framework-facing operations (NCCL EP paper listing, Table V)."""

    def __init__(self, group: Group):
        self.group = group

    def handle(self, num_tokens: int, device=None) -> Handle:
        return Handle(self.group, num_tokens, device)

    def dispatch(self, x: torch.Tensor, topk_idx: torch.Tensor, topk_weights: torch.Tensor | None,
                 handle: Handle | None = None, fp8: bool = False, recv_meta: bool = True,
                 out: torch.Tensor | None = None, stream=None):
        """Dispatch; with ``handle`` None, first plan ``topk_idx`` on a new
        handle for these tokens (a handle passed in must already be planned).
        Returns ``recv_x, recv_i, recv_w, handle, event`` (plus the FP8 scales
        as ``recv_x = (codes, scales)`` when ``fp8``)."""
        T = x.shape[0]
        plan = handle is None
        if plan:
            handle = Handle(self.group, T, x.device)
        rows = handle.recv_rows
        shape = self.group.recv_shape(T)
        H = self.group.hidden
        scales = None
        if fp8:
            recv = out if out is not None else torch.empty(shape, dtype=torch.float8_e4m3fn, device=x.device)
            scales = torch.empty((rows, H // 128), dtype=torch.float32, device=x.device)
        else:
            recv = out if out is not None else torch.empty(shape, dtype=torch.bfloat16, device=x.device)
        ri = torch.empty(rows, dtype=torch.int32, device=x.device) if recv_meta else None
        rw = torch.empty(rows, dtype=torch.float32, device=x.device) if (recv_meta and topk_weights is not None) else None
        if plan:   # the layout and the dispatch together (one launch for small batches)
            ep_plan_dispatch(handle.ptr, topk_idx, x, topk_weights, recv, scales, ri, rw, stream)
        else:
            ep_dispatch(handle.ptr, x, topk_weights, recv, scales, ri, rw, stream)
        ev = _event_on(stream)
        recv_x = (recv, scales) if fp8 else recv
        return recv_x, ri, rw, handle, ev

    def combine(self, expert_out: torch.Tensor, handle: Handle,
                topk_weights: torch.Tensor | None, out_dtype=torch.bfloat16,
                out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        T, H = handle.num_tokens, self.group.hidden
        y = out if out is not None else torch.empty((T, H), dtype=out_dtype, device=expert_out.device)
        ep_combine(handle.ptr, expert_out, topk_weights, y, stream)
        return y

    def dispatch_bwd(self, grad_recv: torch.Tensor, handle: Handle, stream=None) -> torch.Tensor:
        """Gradient of dispatch: sum of each token's received-row gradients."""
        return self.combine(grad_recv, handle, None, stream=stream)

    def combine_bwd(self, grad_y: torch.Tensor, expert_out: torch.Tensor,
                    topk_weights: torch.Tensor, handle: Handle, stream=None):
        grad_out = torch.empty_like(expert_out)
        grad_w = torch.empty_like(topk_weights)
        ep_combine_bwd(handle.ptr, grad_y, expert_out, topk_weights, grad_out, grad_w, stream)
        return grad_out, grad_w

    def prefetch_replicas(self, expert_weights: torch.Tensor, handle: Handle,
                          slots: torch.Tensor | None = None, stream=None,
                          scales: bool | str = False) -> torch.Tensor:
        """Copy the plan's replica experts' weights ([E, P...]) into their
        prefetch slots ([R, S, P...]); slots the plan leaves empty keep their
        contents (uninitialised if ``slots`` is None).  ``scales``: the
        tensor is the fp32 scales of FP8 weights (``"row"``: of INT8 weights)."""
        c = self.group.cfg
        if slots is None:
            slots = torch.empty((c.num_ranks, c.slots_per_rank) + tuple(expert_weights.shape[1:]),
                                dtype=expert_weights.dtype, device=expert_weights.device)
        ep_prefetch_replicas(handle.ptr, expert_weights, slots, stream, scales=scales)
        return slots

    def expert_gemm(self, recv: torch.Tensor, expert_weights: torch.Tensor, handle: Handle,
                    slots: torch.Tensor | None = None, out: torch.Tensor | None = None,
                    stream=None, swiglu: bool = False) -> torch.Tensor:
        """Grouped GEMM of the experts over the received rows: ``recv``
        [rows, K] (any leading shape) times each group's [N, K] weights.
        With ``swiglu`` the weight rows interleave gate (even) and up (odd)
        projections and the result is [rows, N/2] of silu(gate) * up."""
        N = expert_weights.shape[1]
        rows = handle.recv_rows
        if out is None:
            out = torch.empty((rows, N // 2 if swiglu else N), dtype=torch.bfloat16, device=recv.device)
        ep_expert_gemm(handle.ptr, recv.view(rows, expert_weights.shape[2]), expert_weights, slots,
                       out, stream, swiglu=swiglu)
        return out

    def expert_gemm_fp8(self, recv: torch.Tensor, recv_scales: torch.Tensor,
                        expert_weights: torch.Tensor, expert_scales: torch.Tensor, handle: Handle,
                        slots: torch.Tensor | None = None, slot_scales: torch.Tensor | None = None,
                        out: torch.Tensor | None = None, stream=None,
                        swiglu: bool = False) -> torch.Tensor:
        """The grouped GEMM on FP8 operands: ``recv`` e4m3 [rows, K] with fp32
        ``recv_scales`` [rows, K/128] (the FP8 dispatch output), weights e4m3
        [E, N, K] with fp32 scales [E, N, K/128].  ``swiglu`` as in
        ``expert_gemm``."""
        N, K = expert_weights.shape[1], expert_weights.shape[2]
        rows = handle.recv_rows
        if out is None:
            out = torch.empty((rows, N // 2 if swiglu else N), dtype=torch.bfloat16, device=recv.device)
        ep_expert_gemm_fp8(handle.ptr, recv.view(rows, K), recv_scales.view(rows, K // 128),
                           expert_weights, expert_scales, slots, slot_scales, out, stream,
                           swiglu=swiglu)
        return out

    @staticmethod
    def quantize_fp8(x: torch.Tensor, codes: torch.Tensor | None = None,
                     scales: torch.Tensor | None = None, stream=None, pow2: bool = False):
        """bf16 rows [..., K] (K % 128 == 0) to e4m3 codes of the same shape
        and fp32 scales [..., K/128], bit for bit the FP8 dispatch's
        quantisation (``pow2``: power-of-two scales, as a group with
        fp8_scales="pow2"); for the activation between the two FFN GEMMs,
        or for FP8 weights."""
        K = x.shape[-1]
        if codes is None:
            codes = torch.empty(x.shape, dtype=torch.float8_e4m3fn, device=x.device)
        if scales is None:
            scales = torch.empty(tuple(x.shape[:-1]) + (K // 128,), dtype=torch.float32, device=x.device)
        ep_quantize_fp8(x, codes, scales, stream, pow2=pow2)
        return codes, scales

    @staticmethod
    def add_rmsnorm(x: torch.Tensor, residual: torch.Tensor | None, weight: torch.Tensor,
                    eps: float = 1e-6, quant: str = "none", y: bool = True, stream=None):
        """Residual addition and RMS norm of bf16 rows [..., H]: returns
        (hidden, y, codes, scales), None for what was not asked for (hidden is
        x itself without a residual).  ``quant``: "int8", "fp8", "fp8_pow2"."""
        hidden = torch.empty_like(residual) if residual is not None else None
        out = torch.empty_like(x) if y else None
        codes = scales = None
        if quant != "none":
            i8 = quant == "int8"
            codes = torch.empty(x.shape, dtype=torch.int8 if i8 else torch.float8_e4m3fn, device=x.device)
            scales = torch.empty(tuple(x.shape[:-1]) + (() if i8 else (x.shape[-1] // 128,)),
                                 dtype=torch.float32, device=x.device)
        ep_add_rmsnorm(x, residual, weight, hidden, out, codes, scales, eps, quant, stream)
        return x if hidden is None else hidden, out, codes, scales

    @staticmethod
    def add_rmsnorm_bwd(hidden: torch.Tensor, weight: torch.Tensor, grad_y: torch.Tensor,
                        grad_residual_out: torch.Tensor | None = None, eps: float = 1e-6,
                        workspace: torch.Tensor | None = None, stream=None):
        """Gradients (of x and the residual alike, of the weight in fp32)."""
        H = hidden.shape[-1]
        grad = torch.empty_like(hidden)
        gw = torch.empty(H, dtype=torch.float32, device=hidden.device)
        if workspace is None:
            n = ep_add_rmsnorm_bwd_workspace_bytes(hidden.numel() // H, H) // 4
            with torch.cuda.stream(_stream_object(stream)):   # let go of on return: the memory is the call's stream's
                workspace = torch.empty(n, dtype=torch.float32, device=hidden.device)
        ep_add_rmsnorm_bwd(hidden, weight, grad_y, grad_residual_out, grad, gw, workspace, eps, stream)
        return grad, gw

    @staticmethod
    def quantize_int8(x: torch.Tensor, codes: torch.Tensor | None = None,
                      scales: torch.Tensor | None = None, stream=None):
        """bf16 rows [..., K] to int8 codes of the same shape and one fp32
        scale a row; for the activation between the two FFN products, or
        for INT8 weights."""
        if codes is None:
            codes = torch.empty(x.shape, dtype=torch.int8, device=x.device)
        if scales is None:
            scales = torch.empty(x.shape[:-1], dtype=torch.float32, device=x.device)
        ep_quantize_int8(x, codes, scales, stream)
        return codes, scales

    def dispatch_quantized(self, codes: torch.Tensor, scales: torch.Tensor,
                           topk_weights: torch.Tensor | None, handle: Handle,
                           recv_meta: bool = True, stream=None):
        """Dispatch of rows that are 8 bits already (int8 with a scale a row,
        or e4m3 with one per 128 channels) by a planned handle: returns
        ``(recv_codes, recv_scales), recv_i, recv_w, handle, event`` like
        ``dispatch``."""
        rows, dev = handle.recv_rows, codes.device
        recv = torch.empty(self.group.recv_shape(handle.num_tokens), dtype=codes.dtype, device=dev)
        rs = torch.empty((rows,) + tuple(scales.shape[1:]), dtype=torch.float32, device=dev)
        ri = torch.empty(rows, dtype=torch.int32, device=dev) if recv_meta else None
        rw = torch.empty(rows, dtype=torch.float32, device=dev) if recv_meta and topk_weights is not None else None
        ep_dispatch_quantized(handle.ptr, codes, scales, topk_weights, recv, rs, ri, rw, stream)
        ev = _event_on(stream)
        return (recv, rs), ri, rw, handle, ev

    def expert_gemm_int8(self, recv: torch.Tensor, recv_scales: torch.Tensor,
                         expert_weights: torch.Tensor, expert_scales: torch.Tensor, handle: Handle,
                         slots: torch.Tensor | None = None, slot_scales: torch.Tensor | None = None,
                         out: torch.Tensor | None = None, stream=None,
                         swiglu: bool = False) -> torch.Tensor:
        """The grouped GEMM on INT8 operands: ``recv`` int8 [rows, K] with one
        fp32 scale a row, weights int8 [E, N, K] with fp32 scales [E, N].
        ``swiglu`` as in ``expert_gemm``."""
        N, K = expert_weights.shape[1], expert_weights.shape[2]
        rows = handle.recv_rows
        if out is None:
            out = torch.empty((rows, N // 2 if swiglu else N), dtype=torch.bfloat16, device=recv.device)
        ep_expert_gemm_int8(handle.ptr, recv.view(rows, K), recv_scales.view(rows), expert_weights,
                            expert_scales, slots, slot_scales, out, stream, swiglu=swiglu)
        return out

    def dup_grad_reduce(self, replica_grads: torch.Tensor, owner_grads: torch.Tensor,
                        handle: Handle, replica_expert: torch.Tensor | None = None,
                        stream=None) -> torch.Tensor:
        ep_dup_grad_reduce(handle.ptr, replica_grads, replica_expert, owner_grads, stream)
        return owner_grads
