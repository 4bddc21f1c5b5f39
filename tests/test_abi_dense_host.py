"""Host-side refusals of the dense half's entry points (dropout, layer norm and
its backward, block quantiser, FP8 product): every call fails validation before
anything would be enqueued, so no GPU is needed."""

from __future__ import annotations

import ctypes

import pytest
import torch

import combine_ep_plan_amd as ep
from tests.test_abi_front_host import (BF16, DTYPE, EW, F8S, FP32, FP8, I8, I32, INVALID, NW, OK, RS, SHAPE, SMALL,
                                       T_, TAG, UNSUPPORTED, WS, view)
from tests.test_abi_host import FAKE, lib  # noqa: F401  (lib: fixture)

RNG, ST = ep.TAG_RNG_STATE, ep.TAG_STATUS
NAN, INF = float("nan"), float("inf")


def addr(kind, *v):
    return ctypes.byref(kind(*v))


def views(*v):
    return (ctypes.c_void_p * len(v))(*(ctypes.cast(t, ctypes.c_void_p) if t is not None else None for t in v))


@pytest.mark.parametrize("p", [-0.01, 1.01, NAN, INF])
def test_dropout_probability(lib, p):  # noqa: F811
    x = view(BF16, T_, 4, 64)
    assert lib.ep_dropout(addr(ep.ep_dropout_rule_t, p), view(I32, RNG, 4), x, None, x, None) == INVALID
    r = addr(ep.ep_layernorm_rule_t, 1e-5, p, 0, 0)
    io = views(x, None, view(BF16, NW, 64), None, view(I32, RNG, 4), x, x, None, None)
    assert lib.ep_add_layernorm(r, io, None) == INVALID


def test_dropout_refusals(lib):  # noqa: F811
    r = addr(ep.ep_dropout_rule_t, 0.5)
    good = [view(I32, RNG, 4), view(BF16, T_, 4, 64), view(FP32, T_, 4, 64), view(FP32, T_, 4, 64)]
    for at, v, want in [(0, None, INVALID), (0, view(FP32, RNG, 4), DTYPE), (0, view(I32, RNG, 5), SHAPE),
                        (0, view(I32, T_, 4), TAG), (0, view(I32, RNG, 2, 2), SHAPE),
                        (0, view(I32, RNG, 4, data=FAKE + 2), INVALID),
                        (1, None, INVALID), (1, view(FP8, T_, 4, 64), DTYPE), (1, view(BF16, T_, 4, 60), SHAPE),
                        (1, view(BF16, T_, 64), SHAPE), (1, view(BF16, T_, 4, 64, data=FAKE + 8), INVALID),
                        (2, view(BF16, T_, 4, 64), DTYPE), (2, view(FP32, T_, 5, 64), SHAPE),
                        (3, None, INVALID), (3, view(I32, T_, 4, 64), DTYPE), (3, view(FP32, T_, 4, 72), SHAPE),
                        (3, view(FP32, NW, 4, 64), TAG)]:
        a = list(good)
        a[at] = v
        assert lib.ep_dropout(r, *a, None) == want, (at, want)
    assert lib.ep_dropout(None, *good, None) == INVALID


def _rule(eps=1e-5, p=0.0, quant=0, reserved=0):
    return addr(ep.ep_layernorm_rule_t, eps, p, quant, reserved)


@pytest.mark.parametrize("bad", [dict(eps=0.0), dict(eps=-1.0), dict(eps=NAN), dict(eps=INF), dict(eps=1e-39),
                                 dict(quant=4), dict(quant=-1), dict(reserved=1)])
def test_layernorm_rules(lib, bad):  # noqa: F811
    x, w = view(BF16, T_, 4, 128), view(BF16, NW, 128)
    q = bad.get("quant", 0)
    io = views(x, None, w, None, None, None, x, view(FP8, T_, 4, 128) if q else None, view(FP32, F8S, 4, 1) if q else None)
    assert lib.ep_add_layernorm(_rule(**bad), io, None) == INVALID
    bwd = views(x, w, x, None, None, x, None, None, None, None)
    assert lib.ep_add_layernorm_bwd(_rule(**bad), bwd, None) == INVALID
    assert lib.ep_add_layernorm(None, io, None) == INVALID and lib.ep_add_layernorm(_rule(), None, None) == INVALID
    assert lib.ep_add_layernorm_bwd(None, bwd, None) == INVALID and lib.ep_add_layernorm_bwd(_rule(), None, None) == INVALID
    assert lib.ep_add_layernorm_bwd(_rule(quant=1), bwd, None) == INVALID


def test_layernorm_refusals(lib):  # noqa: F811
    """Members: x, residual, weight, bias, rng, residual_out, y, codes, scales."""
    x, f = view(BF16, T_, 4, 128), view(FP32, T_, 4, 128)
    w, g = view(BF16, NW, 128), view(I32, RNG, 4)
    good = [x, f, w, w, g, f, x, view(FP8, T_, 4, 128), view(FP32, F8S, 4, 1)]
    for at, v, want in [(0, None, INVALID), (0, f, DTYPE), (0, view(BF16, T_, 4, 124), SHAPE),
                        (0, view(BF16, T_, 4, 32776), UNSUPPORTED), (1, view(FP8, T_, 4, 128), DTYPE),
                        (1, x, DTYPE), (1, view(FP32, T_, 3, 128), SHAPE), (2, None, INVALID),
                        (2, view(BF16, NW, 120), SHAPE), (2, view(FP32, NW, 128), DTYPE), (2, view(BF16, T_, 128), TAG),
                        (3, view(FP32, NW, 128), DTYPE), (3, view(BF16, NW, 64), SHAPE), (4, None, INVALID),
                        (4, view(I32, RNG, 2), SHAPE), (5, None, INVALID), (5, x, DTYPE), (6, f, DTYPE),
                        (6, view(BF16, T_, 128, 4), SHAPE), (7, None, INVALID), (7, view(I8, T_, 4, 128), DTYPE),
                        (8, None, INVALID), (8, view(FP32, RS, 4), TAG), (8, view(FP32, F8S, 4, 2), SHAPE)]:
        a = list(good)
        a[at] = v
        assert lib.ep_add_layernorm(_rule(p=0.5, quant=1), views(*a), None) == want, (at, want)
    none = [x, None, w, None, None, None, x, None, None]
    for at, v in [(4, g), (5, x), (7, view(FP8, T_, 4, 128)), (6, None)]:   # a state or stream that nothing asks for
        a = list(none)
        a[at] = v
        assert lib.ep_add_layernorm(_rule(), views(*a), None) == INVALID, at
    a = [x, None, w, None, g, f, x, None, None]   # without a residual the stream is bf16
    assert lib.ep_add_layernorm(_rule(p=0.5), views(*a), None) == DTYPE
    x8 = view(BF16, T_, 4, 64)
    a = [x8, None, view(BF16, NW, 64), None, None, None, x8, view(FP8, T_, 4, 64), view(FP32, F8S, 4, 1)]
    assert lib.ep_add_layernorm(_rule(quant=1), views(*a), None) == UNSUPPORTED


def test_layernorm_bwd_refusals(lib):  # noqa: F811
    """Members: hidden, weight, grad_y, grad_residual_out, rng, grad, grad_x, grad_weight, grad_bias, workspace."""
    x, f = view(BF16, T_, 4, 128), view(FP32, T_, 4, 128)
    w, g, d = view(BF16, NW, 128), view(I32, RNG, 4), view(FP32, NW, 128)
    good = [f, w, x, f, g, f, x, d, d, view(FP32, WS, 1 << 16)]
    for at, v, want in [(0, None, INVALID), (0, view(FP8, T_, 4, 128), DTYPE), (0, view(FP32, T_, 4, 32776), UNSUPPORTED),
                        (1, None, INVALID), (1, view(BF16, NW, 64), SHAPE), (2, None, INVALID), (2, f, DTYPE),
                        (2, view(BF16, T_, 5, 128), SHAPE), (3, x, DTYPE), (4, None, INVALID), (5, x, DTYPE),
                        (6, None, INVALID), (6, f, DTYPE), (7, view(BF16, NW, 128), DTYPE), (8, view(FP32, NW, 64), SHAPE),
                        (9, None, INVALID), (9, view(FP32, WS, 8), SMALL), (9, view(FP32, WS, 8, 1 << 13), SHAPE),
                        (9, view(FP32, T_, 1 << 16), TAG)]:
        a = list(good)
        a[at] = v
        assert lib.ep_add_layernorm_bwd(_rule(p=0.5), views(*a), None) == want, (at, want)
    a = [f, w, x, f, None, None, None, d, d, view(FP32, WS, 1 << 16)]
    assert lib.ep_add_layernorm_bwd(_rule(), views(*a), None) == INVALID   # no gradient asked for
    a[5], a[6] = f, x
    assert lib.ep_add_layernorm_bwd(_rule(), views(*a), None) == INVALID   # grad_x without dropout
    n = ctypes.c_size_t()
    for rows, H in [(-1, 64), (4, 0), (4, 12), (4, 32776), (1 << 31, 64)]:
        assert lib.ep_add_layernorm_bwd_workspace_bytes(rows, H, ctypes.byref(n)) == INVALID
    assert lib.ep_add_layernorm_bwd_workspace_bytes(0, 64, ctypes.byref(n)) == OK and n.value == 0
    m = ctypes.c_size_t()
    assert lib.ep_add_layernorm_bwd_workspace_bytes(700, 64, ctypes.byref(n)) == OK
    assert lib.ep_add_rmsnorm_bwd_workspace_bytes(700, 64, ctypes.byref(m)) == OK and n.value == 2 * m.value > 0


def test_quantize_2d_refusals(lib):  # noqa: F811
    rows, square = addr(ep.ep_fp8_2d_rule_t, 0, 0), addr(ep.ep_fp8_2d_rule_t, 1, 1)
    x = view(BF16, T_, 130, 256)
    c, ct = view(FP8, T_, 130, 256), view(FP8, T_, 256, 256)
    good = [x, c, view(FP32, F8S, 130, 2), ct, view(FP32, F8S, 256, 2)]
    for at, v, want in [(0, None, INVALID), (0, view(FP32, T_, 130, 256), DTYPE), (0, view(BF16, T_, 130, 200), SHAPE),
                        (0, view(BF16, T_, 2, 65, 256), SHAPE), (1, None, INVALID), (1, view(I8, T_, 130, 256), DTYPE),
                        (1, view(FP8, T_, 128, 256), SHAPE), (2, None, INVALID), (2, view(FP32, F8S, 2, 2), SHAPE),
                        (2, view(FP32, RS, 130, 2), TAG), (3, None, INVALID), (3, view(FP8, T_, 256, 130), SHAPE),
                        (4, None, INVALID), (4, view(FP32, F8S, 2, 2), SHAPE)]:
        a = list(good)
        a[at] = v
        assert lib.ep_quantize_fp8_2d(rows, *a, None) == want, (at, want)
    a = [x, c, view(FP32, F8S, 130, 2), None, None]
    assert lib.ep_quantize_fp8_2d(square, *a, None) == SHAPE
    assert lib.ep_quantize_fp8_2d(rows, x, None, None, None, None, None) == INVALID
    for bad in ((2, 0), (-1, 0), (0, 2), (0, -1)):
        assert lib.ep_quantize_fp8_2d(addr(ep.ep_fp8_2d_rule_t, *bad), *good, None) == INVALID
    assert lib.ep_quantize_fp8_2d(None, *good, None) == INVALID
    R, C = 1 << 19, 1 << 19
    a = [view(BF16, T_, R, C), view(FP8, T_, R, C), view(FP32, F8S, R, C // 128), None, None]
    assert lib.ep_quantize_fp8_2d(rows, *a, None) == UNSUPPORTED


def test_linear_refusals(lib):  # noqa: F811
    rule = lambda s=0, g=0: addr(ep.ep_linear_rule_t, s, g)  # noqa: E731
    x, w = view(FP8, T_, 5, 256), view(FP8, EW, 130, 256)
    out = view(FP32, T_, 5, 130)
    good = [x, view(FP32, F8S, 5, 2), w, view(FP32, F8S, 2, 2), out, out, view(I32, ST, 1)]
    for at, v, want in [(0, None, INVALID), (0, view(BF16, T_, 5, 256), DTYPE), (0, view(FP8, T_, 5, 200), SHAPE),
                        (0, view(FP8, T_, 5, 384), SHAPE), (0, view(FP8, T_, 5, 0), SHAPE), (0, view(FP8, T_, 256), SHAPE), (1, None, INVALID),
                        (1, view(FP32, F8S, 5, 3), SHAPE), (1, view(FP32, RS, 5, 2), TAG), (2, None, INVALID),
                        (2, view(FP8, T_, 130, 256), TAG), (2, view(FP8, EW, 1, 130, 256), SHAPE),
                        (2, view(BF16, EW, 130, 256), DTYPE), (3, view(FP32, F8S, 3, 2), SHAPE),
                        (3, view(FP32, F8S, 1, 2), SHAPE), (3, None, INVALID), (4, view(BF16, T_, 5, 130), DTYPE),
                        (4, view(FP32, T_, 5, 128), SHAPE), (5, None, INVALID), (5, view(FP8, T_, 5, 130), DTYPE),
                        (5, view(FP32, T_, 130, 5), SHAPE), (6, view(FP32, ST, 1), DTYPE), (6, view(I32, ST, 2), SHAPE),
                        (6, view(I32, RNG, 1), TAG)]:
        a = list(good)
        a[at] = v
        assert lib.ep_linear_fp8(rule(), *a, None) == want, (at, want)
    assert lib.ep_linear_fp8(None, *good, None) == INVALID
    for bad in ((2, 0), (-1, 0), (0, 2), (0, -1)):
        assert lib.ep_linear_fp8(rule(*bad), *good, None) == INVALID
    w, half = view(FP8, EW, 32, 256), view(BF16, T_, 5, 16)
    glu = [x, view(FP32, F8S, 5, 2), w, view(FP32, F8S, 1, 2), None, half, None]
    for at, v, want in [(4, half, INVALID), (5, view(FP32, T_, 5, 16), DTYPE), (5, view(BF16, T_, 5, 32), SHAPE),
                        (2, view(FP8, EW, 40, 256), SHAPE)]:
        a = list(glu)
        a[at] = v
        assert lib.ep_linear_fp8(rule(0, 1), *a, None) == want, (at, want)
    K = (1 << 22) + 128
    a = [view(FP8, T_, 5, K), view(FP32, F8S, 5, K // 128), view(FP8, EW, 130, K), view(FP32, F8S, 2, K // 128), None, out, None]
    assert lib.ep_linear_fp8(rule(), *a, None) == UNSUPPORTED
    M = N = (1 << 20)   # 2^28 tiles of 64 x 64
    a = [view(FP8, T_, M, 128), view(FP32, F8S, M, 1), view(FP8, EW, N, 128), view(FP32, F8S, N // 128, 1), None,
         view(BF16, T_, M, N), None]
    assert lib.ep_linear_fp8(rule(), *a, None) == UNSUPPORTED
    N = (1 << 30)   # more than 2^32 threads of the few tokens' kernel
    a = [view(FP8, T_, 1, 128), view(FP32, F8S, 1, 1), view(FP8, EW, N, 128), view(FP32, F8S, N // 128, 1), None,
         view(BF16, T_, 1, N), None]
    assert lib.ep_linear_fp8(rule(), *a, None) == UNSUPPORTED


def test_the_binding_refuses_what_is_not_on_the_gpu():
    x = torch.zeros(4, 128, dtype=torch.bfloat16)
    w = torch.ones(128)
    rng = torch.zeros(4, dtype=torch.int32)
    with pytest.raises((ValueError, RuntimeError)):
        ep.Buffer.dropout(x, 0.5, rng)
    with pytest.raises((ValueError, RuntimeError)):
        ep.Buffer.add_layernorm(x, None, w)
    with pytest.raises((ValueError, RuntimeError)):
        ep.Buffer.quantize_fp8_2d(x)


def test_rng_state_words():
    s = ep.rng_state((1 << 63) + 5, (3 << 32) + 0xFFFFFFFF, device="cpu")
    assert s.dtype == torch.int32 and s.tolist() == [5, -2 ** 31, -1, 3]


def test_recorded_calls_reach_the_entry_points(lib):  # noqa: F811
    """ep_run_calls hands each op its own arguments: a refusal of the entry point comes back."""
    x = view(BF16, T_, 4, 64)
    cast = lambda v: ctypes.cast(v, ctypes.c_void_p).value  # noqa: E731
    io = views(x, None, view(BF16, NW, 64), None, None, None, None, None, None)
    ln, dr = ep.ep_layernorm_rule_t(1e-5, 0.0, 0, 0), ep.ep_dropout_rule_t(2.0)
    q2, li = ep.ep_fp8_2d_rule_t(0, 0), ep.ep_linear_rule_t(0, 0)
    bwd = views(x, view(BF16, NW, 60), x, None, None, x, None, None, None, None)
    calls = [(23, [ctypes.addressof(dr), cast(view(I32, RNG, 4)), cast(x), None, cast(x)], INVALID),
             (24, [ctypes.addressof(ln), ctypes.addressof(io)], INVALID),
             (25, [ctypes.addressof(ln), ctypes.addressof(bwd)], SHAPE),
             (26, [ctypes.addressof(q2), cast(x), cast(x), cast(x), None, None], SHAPE),
             (27, [ctypes.addressof(li), cast(x), cast(x), cast(x), cast(x), None, cast(x), None], DTYPE),
             (28, [], INVALID)]
    for op, p, want in calls:
        c = ep.ep_call_t()
        c.op = op
        for i, v in enumerate(p):
            c.p[i] = v
        failed = ctypes.c_int32(-1)
        assert lib.ep_run_calls(ctypes.byref(c), 1, ctypes.byref(failed)) == want, op
        assert failed.value == 0
