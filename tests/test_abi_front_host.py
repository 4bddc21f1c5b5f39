"""Host-side refusals of the MoE front's entry points (scored routing, RMS
norm, 8-bit rows, INT8 GEMM): every call fails validation before anything
would be enqueued, so no GPU is needed."""

from __future__ import annotations

import ctypes

import pytest
import torch

import combine_ep_plan_amd as ep
from tests.test_abi_host import FAKE, create, lib  # noqa: F401  (lib: fixture)

OK, INVALID, TAG, DTYPE, SHAPE, UNPLANNED, SMALL, UNSUPPORTED = 0, 1, 2, 3, 4, 5, 6, 7
BF16, FP32, FP8, I32, I8 = 0, 1, 2, 3, 4
T_, IDX, WTS, F8S, LOG, EW, RS, BIAS, NW, WS = (ep.TAG_TOKENS, ep.TAG_TOPK_IDX, ep.TAG_TOPK_WEIGHTS,
                                                ep.TAG_FP8_SCALES, ep.TAG_ROUTER_LOGITS,
                                                ep.TAG_EXPERT_WEIGHTS, ep.TAG_ROW_SCALES,
                                                ep.TAG_ROUTER_BIAS, ep.TAG_NORM_WEIGHT,
                                                ep.TAG_WORKSPACE)


def view(dtype, tag, *sizes, data=FAKE):
    return ctypes.pointer(ep.ep_tensor_t(data, dtype, tag, len(sizes), 0, (ctypes.c_int64 * 4)(*sizes)))


def handle(lib, T=16, **kw):  # noqa: F811
    rc, g = create(lib, **kw)
    assert rc == OK
    h = ctypes.c_void_p()
    assert lib.ep_handle_create(g, T, FAKE, 1 << 30, ctypes.byref(h)) == OK
    return h


def rule(**kw):
    base = dict(score="sigmoid", num_groups=4, kept_groups=2, group_score="top2")
    base.update(kw)
    return ep.RouteRule(**base).ptr


BAD_RULES = [dict(score=2), dict(score=-1), dict(num_groups=0), dict(num_groups=3), dict(num_groups=65),
             dict(kept_groups=0), dict(kept_groups=5), dict(group_score=2), dict(renormalise=2),
             dict(scale=float("nan")), dict(scale=float("inf"))]


@pytest.mark.parametrize("bad", BAD_RULES)
def test_route_rules(lib, bad):  # noqa: F811
    h = handle(lib)
    lg, i, w = view(FP32, LOG, 16, 8), view(I32, IDX, 16, 2), view(FP32, WTS, 16, 2)
    assert lib.ep_route_scored(h, rule(**bad), lg, None, i, w, None, None) == INVALID
    assert lib.ep_route_scored_bwd(h, rule(**bad), lg, i, w, None, lg, None) == INVALID


def test_route_refusals(lib):  # noqa: F811
    h, r = handle(lib), rule()
    good = [view(FP32, LOG, 16, 8), view(FP32, BIAS, 8), view(I32, IDX, 16, 2), view(FP32, WTS, 16, 2),
            view(FP32, LOG, 16, 8)]
    call = lambda *a: lib.ep_route_scored(h, r, *a, None)  # noqa: E731
    for at, v, want in [(0, view(I32, LOG, 16, 8), DTYPE), (0, view(FP32, T_, 16, 8), TAG),
                        (0, view(FP32, LOG, 15, 8), SHAPE), (0, None, INVALID),
                        (0, view(FP32, LOG, 16, 8, data=FAKE + 2), INVALID),
                        (1, view(BF16, BIAS, 8), DTYPE), (1, view(FP32, BIAS, 7), SHAPE),
                        (1, view(FP32, WTS, 8), TAG), (2, view(I32, IDX, 16, 3), SHAPE), (2, None, INVALID),
                        (3, view(BF16, WTS, 16, 2), DTYPE), (4, view(BF16, LOG, 16, 8), DTYPE),
                        (4, view(FP32, LOG, 8, 16), SHAPE)]:
        a = list(good)
        a[at] = v
        assert call(*a) == want, (at, want)
    assert lib.ep_route_scored(None, r, *good, None) == INVALID
    assert lib.ep_route_scored(h, None, *good, None) == INVALID
    bf = view(BF16, LOG, 16, 8)   # the gradient has the logits' dtype
    assert lib.ep_route_scored_bwd(h, r, bf, good[2], good[3], None, good[0], None) == DTYPE
    assert lib.ep_route_scored_bwd(h, r, bf, good[2], good[3], bf, bf, None) == DTYPE


def test_route_refuses_launches_past_32_bits(lib):  # noqa: F811
    T = 1 << 26
    rc, g = create(lib, hidden=64, max_tokens=T)
    assert rc == OK
    h = ctypes.c_void_p()
    assert lib.ep_handle_create(g, T, FAKE, 1 << 36, ctypes.byref(h)) == OK
    lg, i, w = view(FP32, LOG, T, 8), view(I32, IDX, T, 2), view(FP32, WTS, T, 2)
    assert lib.ep_route_scored(h, rule(), lg, None, i, w, None, None) == UNSUPPORTED
    assert lib.ep_route_scored_bwd(h, rule(), lg, i, w, None, lg, None) == UNSUPPORTED


def norm_rule(eps=1e-6, quant=0, reserved=0):
    return ctypes.pointer(ep.ep_norm_rule_t(eps, quant, reserved))


def test_norm_refusals(lib):  # noqa: F811
    x, w, y = view(BF16, T_, 4, 256), view(BF16, NW, 256), view(BF16, T_, 4, 256)
    q8, s8 = view(I8, T_, 4, 256), view(FP32, RS, 4)
    qf, sf = view(FP8, T_, 4, 256), view(FP32, F8S, 4, 2)
    f = lib.ep_add_rmsnorm
    for bad in (norm_rule(0.0), norm_rule(-1.0), norm_rule(float("nan")), norm_rule(float("inf")), norm_rule(1e-39),
                norm_rule(quant=4), norm_rule(quant=-1), norm_rule(reserved=1), None):
        assert f(bad, x, None, w, None, y, None, None, None) == INVALID
    r = norm_rule()
    assert f(r, x, None, w, None, None, None, None, None) == INVALID          # no output
    assert f(r, x, x, w, None, y, None, None, None) == INVALID                # residual without its sum
    assert f(r, x, None, w, y, y, None, None, None) == INVALID
    assert f(r, x, None, w, None, y, q8, s8, None) == INVALID                 # codes without a format
    assert f(norm_rule(quant=3), x, None, w, None, y, None, None, None) == INVALID
    assert f(norm_rule(quant=3), x, None, w, None, y, q8, None, None) == INVALID
    assert f(norm_rule(quant=3), x, None, w, None, y, qf, s8, None) == DTYPE
    assert f(norm_rule(quant=3), x, None, w, None, y, q8, sf, None) == TAG
    assert f(norm_rule(quant=3), x, None, w, None, y, q8, view(FP32, RS, 5), None) == SHAPE
    assert f(norm_rule(quant=1), x, None, w, None, y, qf, view(FP32, F8S, 4, 3), None) == SHAPE
    assert f(norm_rule(quant=1), x, None, w, None, y, q8, sf, None) == DTYPE
    x2 = view(BF16, T_, 4, 136)
    assert f(norm_rule(quant=1), x2, None, view(BF16, NW, 136), None, None, view(FP8, T_, 4, 136),
             view(FP32, F8S, 4, 1), None) == UNSUPPORTED
    assert f(r, view(FP32, T_, 4, 256), None, w, None, y, None, None, None) == DTYPE
    assert f(r, view(BF16, T_, 4, 252), None, w, None, y, None, None, None) == SHAPE
    assert f(r, view(BF16, T_, 256), None, w, None, y, None, None, None) == SHAPE
    assert f(r, x, None, view(BF16, NW, 128), None, y, None, None, None) == SHAPE
    assert f(r, x, None, view(BF16, T_, 256), None, y, None, None, None) == TAG
    assert f(r, x, None, view(BF16, NW, 256, data=FAKE + 8), None, y, None, None, None) == INVALID
    assert f(r, x, view(BF16, T_, 4, 256), w, view(FP32, T_, 4, 256), y, None, None, None) == DTYPE
    assert f(r, x, view(BF16, T_, 3, 256), w, view(BF16, T_, 4, 256), y, None, None, None) == SHAPE
    big = 32776
    assert f(r, view(BF16, T_, 4, big), None, view(BF16, NW, big), None, view(BF16, T_, 4, big), None,
             None, None) == UNSUPPORTED
    assert f(r, view(BF16, T_, 1 << 31, 8), None, view(BF16, NW, 8), None, view(BF16, T_, 1 << 31, 8),
             None, None, None) == SHAPE


def test_norm_bwd_refusals(lib):  # noqa: F811
    f, r = lib.ep_add_rmsnorm_bwd, norm_rule()
    h, w, gw = view(BF16, T_, 4, 256), view(BF16, NW, 256), view(FP32, NW, 256)
    need = ctypes.c_size_t()
    assert lib.ep_add_rmsnorm_bwd_workspace_bytes(4, 256, ctypes.byref(need)) == OK
    assert 256 * 4 <= need.value <= 4 * 256 * 4   # at least one partial row, at most one a row
    n = need.value // 4
    for rows, H in ((-1, 256), (4, 0), (4, 12), (4, 32776), (1 << 31, 256)):
        assert lib.ep_add_rmsnorm_bwd_workspace_bytes(rows, H, ctypes.byref(need)) == INVALID
    ws = view(FP32, WS, n)
    assert f(norm_rule(quant=1), h, w, h, None, h, gw, ws, None) == INVALID
    assert f(r, None, w, h, None, h, gw, ws, None) == INVALID
    assert f(r, h, w, h, None, h, gw, None, None) == INVALID
    assert f(r, h, w, h, None, h, gw, view(FP32, WS, n - 1), None) == SMALL
    assert f(r, h, w, h, None, h, gw, view(FP32, WS, 4, 256), None) == SHAPE
    assert f(r, h, w, h, None, h, gw, view(FP32, T_, n), None) == TAG
    assert f(r, h, w, h, None, h, view(BF16, NW, 256), ws, None) == DTYPE
    assert f(r, h, w, view(FP32, T_, 4, 256), None, h, gw, ws, None) == DTYPE
    assert f(r, h, w, h, view(FP32, T_, 4, 256), h, gw, ws, None) == DTYPE
    assert f(r, h, w, h, None, view(FP32, T_, 4, 256), gw, ws, None) == DTYPE
    assert f(r, h, w, view(BF16, T_, 5, 256), None, h, gw, ws, None) == SHAPE


def test_quantize_int8_refusals(lib):  # noqa: F811
    f = lib.ep_quantize_int8
    x, q, s = view(BF16, T_, 4, 64), view(I8, T_, 4, 64), view(FP32, RS, 4)
    for a, want in [((None, q, s), INVALID), ((view(FP32, T_, 4, 64), q, s), DTYPE),
                    ((x, view(FP8, T_, 4, 64), s), DTYPE), ((x, q, view(FP32, F8S, 4)), TAG),
                    ((x, view(I8, T_, 4, 32), s), SHAPE), ((x, q, view(FP32, RS, 3)), SHAPE),
                    ((view(BF16, T_, 4, 60), view(I8, T_, 4, 60), s), SHAPE),
                    ((view(BF16, T_, 4, 32776), view(I8, T_, 4, 32776), s), UNSUPPORTED),
                    ((view(BF16, T_, 4, 64, data=FAKE + 8), q, s), INVALID)]:
        assert f(*a, None) == want


def test_dispatch_quantized_refusals(lib):  # noqa: F811
    h = handle(lib)            # H 256, T 16, k 2: 32 receive rows
    f = lib.ep_dispatch_quantized
    x, s, o, so = view(I8, T_, 16, 256), view(FP32, RS, 16), view(I8, T_, 32, 256), view(FP32, RS, 32)
    xf, sf, of, sof = (view(FP8, T_, 16, 256), view(FP32, F8S, 16, 2), view(FP8, T_, 32, 256),
                       view(FP32, F8S, 32, 2))
    n = None
    for a, want in [((n, s, n, o, so, n, n), INVALID), ((view(BF16, T_, 16, 256), s, n, o, so, n, n), DTYPE),
                    ((x, sf, n, o, so, n, n), TAG), ((xf, s, n, of, sof, n, n), TAG),
                    ((x, s, n, of, so, n, n), DTYPE), ((x, s, n, o, sof, n, n), TAG),
                    ((x, view(FP32, RS, 15), n, o, so, n, n), SHAPE),
                    ((x, s, n, view(I8, T_, 31, 256), so, n, n), SHAPE),
                    ((xf, sf, n, of, view(FP32, F8S, 32, 3), n, n), SHAPE),
                    ((x, s, n, o, so, n, view(FP32, WTS, 32)), INVALID),   # row weights without weights
                    ((x, s, n, o, so, view(I32, IDX, 31), n), SHAPE),
                    ((x, s, n, o, so, n, n), UNPLANNED)]:
        assert f(h, *a, None) == want
    h8 = handle(lib, hidden=264)   # a multiple of 8, not of 16
    assert f(h8, view(I8, T_, 16, 264), s, n, view(I8, T_, 32, 264), so, n, n, None) == UNSUPPORTED
    h16 = handle(lib, hidden=272)
    assert f(h16, view(FP8, T_, 16, 272), view(FP32, F8S, 16, 2), n, view(FP8, T_, 32, 272),
             view(FP32, F8S, 32, 2), n, n, None) == UNSUPPORTED


@pytest.mark.parametrize("name", ["ep_expert_gemm_int8", "ep_expert_gemm_int8_swiglu"])
def test_gemm_int8_refusals(lib, name):  # noqa: F811
    f, glu = getattr(lib, name), name.endswith("swiglu")
    h = handle(lib)
    K, N = 128, 32
    x, s, w, ws = view(I8, T_, 32, K), view(FP32, RS, 32), view(I8, EW, 8, N, K), view(FP32, RS, 8, N)
    o = view(BF16, T_, 32, N // 2 if glu else N)
    n = None
    wk = lambda k: (view(I8, T_, 32, k), s, view(I8, EW, 8, N, k), ws, n, n, o)  # noqa: E731
    for a, want in [((n, s, w, ws, n, n, o), INVALID), ((view(FP8, T_, 32, K), s, w, ws, n, n, o), DTYPE),
                    ((x, view(FP32, F8S, 32), w, ws, n, n, o), TAG),
                    ((x, s, view(FP8, EW, 8, N, K), ws, n, n, o), DTYPE),
                    ((x, s, view(I8, T_, 8, N, K), ws, n, n, o), TAG),
                    ((x, s, w, view(FP32, RS, 8, N + 1), n, n, o), SHAPE),
                    ((x, view(FP32, RS, 31), w, ws, n, n, o), SHAPE),
                    ((x, s, w, ws, n, n, view(BF16, T_, 32, N + 16)), SHAPE),
                    ((x, s, w, ws, n, n, view(FP32, T_, 32, N)), DTYPE),
                    (wk(96), SHAPE), (wk(131072), UNSUPPORTED),
                    ((x, s, w, ws, w, n, o), INVALID),                       # slots without their scales
                    ((x, s, w, ws, view(I8, EW, 4, N, K), view(FP32, RS, 4, N), o), UNSUPPORTED),
                    ((x, s, w, ws, n, n, o), UNPLANNED)]:
        assert f(h, *a, None) == want
    if glu:
        w24, o12 = view(I8, EW, 8, 24, K), view(BF16, T_, 32, 12)
        assert f(h, x, s, w24, view(FP32, RS, 8, 24), n, n, o12, None) == SHAPE
    wide = 1 << 30   # a grid beyond 32-bit thread counts
    assert f(h, x, s, view(I8, EW, 8, wide, K), view(FP32, RS, 8, wide), n, n,
             view(BF16, T_, 32, wide // 2 if glu else wide), None) == UNSUPPORTED


def test_prefetch_takes_int8_and_row_scales(lib):  # noqa: F811
    h = handle(lib, layout=ep.LAYOUT_STATIC, slots_per_rank=2)
    f = lib.ep_prefetch_replicas
    assert f(h, view(I8, EW, 8, 4, 64), view(I8, EW, 4, 2, 4, 64), None) == UNPLANNED
    assert f(h, view(FP32, RS, 8, 4), view(FP32, RS, 4, 2, 4), None) == UNPLANNED
    assert f(h, view(BF16, RS, 8, 4), view(BF16, RS, 4, 2, 4), None) == DTYPE
    assert f(h, view(FP32, RS, 8, 4), view(FP32, F8S, 4, 2, 4), None) == TAG


def test_recorded_front_calls_check_like_their_entry_points(lib):  # noqa: F811
    """The recorded forms reach the same checks with the same arguments."""
    h, r = handle(lib), rule()
    lg, i, w = view(FP32, LOG, 16, 8), view(I32, IDX, 16, 2), view(FP32, WTS, 16, 2)
    x, s, o, so = view(I8, T_, 16, 256), view(FP32, RS, 16), view(I8, T_, 32, 256), view(FP32, RS, 32)
    wq, ws = view(I8, EW, 8, 32, 256), view(FP32, RS, 8, 32)
    bad = view(FP32, LOG, 15, 8)
    calls = [(15, (h, r, bad, None, i, w, None, None), SHAPE),
             (16, (h, r, lg, i, w, None, bad, None), SHAPE),
             (17, (norm_rule(), view(BF16, T_, 4, 256), None, view(BF16, NW, 128), None,
                   view(BF16, T_, 4, 256), None, None, None), SHAPE),
             (18, (norm_rule(), view(BF16, T_, 4, 256), view(BF16, NW, 256), view(BF16, T_, 4, 256), None,
                   view(BF16, T_, 5, 256), None, None, None), SHAPE),
             (19, (view(BF16, T_, 4, 64), view(I8, T_, 4, 64), view(FP32, RS, 3), None), SHAPE),
             (20, (h, x, s, None, o, so, None, None, None), UNPLANNED),
             (21, (h, o, so, wq, ws, None, None, view(BF16, T_, 32, 32), None), UNPLANNED),
             (22, (h, o, so, wq, ws, None, None, view(BF16, T_, 32, 16), None), UNPLANNED)]
    for op, args, want in calls:
        c = ep.ep_call_t(op, 0)
        for m, a in enumerate(args):
            c.p[m] = None if a is None else ctypes.cast(a, ctypes.c_void_p).value
        assert lib.ep_run_calls(ctypes.byref(c), 1, None) == want, op


def test_marshalling_refuses_what_the_library_cannot_take(lib):  # noqa: F811
    """The C++ marshalling: CPU tensors, non-tensors, a wrong number of
    arguments -- Python errors, nothing called."""
    fn = ep._entry["ep_quantize_int8"]
    x, q, s = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(4, 64, dtype=torch.int8), torch.zeros(4)
    with pytest.raises(ValueError, match="on the GPU"):
        ep._marshal_call(fn, ep._TAGS_QUANTIZE, (0, 0), x, q, s)
    with pytest.raises(TypeError, match="torch.Tensor"):
        ep._marshal_call(fn, ep._TAGS_QUANTIZE, (0, 0), 5, q, s)
    with pytest.raises(TypeError, match="one tag"):
        ep._marshal_call(fn, ep._TAGS_QUANTIZE, (0, 0), x, q)
    with pytest.raises(TypeError, match="stream"):
        ep._marshal_call(fn, ep._TAGS_QUANTIZE, 7, x, q, s)
    # NULL arguments reach the entry point's own checks
    assert ep._marshal_call(fn, ep._TAGS_QUANTIZE, (0, 0), None, None, None) == INVALID
