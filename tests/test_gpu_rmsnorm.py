"""GPU parity of the residual RMS norm, its 8-bit outputs and its backward.

Codes and scales are bit for bit those of the formulas evaluated in fp32
from the once-rounded 1/sqrt; every value is also held against the 64-bit
form: y by two products and two roundings (4 half steps of fp32) and its
own type's rounding, INT8 by half a step, FP8 by half a step of e4m3."""

from __future__ import annotations

import numpy as np
import pytest
import torch

import combine_ep_plan_amd as ep
from oracle import front
from tests.gpu_util import host

pytestmark = pytest.mark.gpu
U, UB = 2.0 ** -24, 2.0 ** -8
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    ep.load_library()


def _rows(rng, T, H, dtype, std=1.0):
    x = rng.normal(size=(T, H)) * std * np.exp(rng.normal(size=H) * 0.5)
    return torch.from_numpy(x.astype(np.float32)).to(dtype).cuda()


SHAPES = [(1, 8), (3, 128), (2, 512), (5, 520), (4, 1024), (1, 7168), (130, 256), (33, 4096), (2, 8192),
          (2, 8200), (3, 16384), (2, 32768), (700, 384)]


@pytest.mark.parametrize("T,H", SHAPES)
@pytest.mark.parametrize("residual", [None, torch.bfloat16, torch.float32])
@pytest.mark.parametrize("quant", ["none", "int8", "fp8", "fp8_pow2"])
def test_add_rmsnorm(T, H, residual, quant):
    if quant.startswith("fp8") and H % 128:
        H = (H + 127) // 128 * 128 if H < 32768 else H
    rng = np.random.default_rng(T * 31 + H)
    x = _rows(rng, T, H, torch.bfloat16)
    r = None if residual is None else _rows(rng, T, H, residual, 2.0)
    w = torch.from_numpy((1 + 0.3 * rng.normal(size=H)).astype(np.float32)).cuda()
    if T % 2:
        w = w.to(torch.bfloat16)
    if T > 2:
        x[T // 2] = 0
        if r is not None:
            r[T // 2] = 0
    want_y = quant in ("none", "fp8")
    hidden, y, codes, scales = ep.Buffer.add_rmsnorm(x, r, w, EPS, quant, y=want_y)
    h_ref = x if r is None else (x.float() + r.float()).to(residual)
    assert torch.equal(hidden, h_ref)
    hn, wn = host(h_ref.float()), host(w.float())
    y64, y32 = front.rmsnorm(hn, wn, EPS)
    if want_y:
        assert torch.equal(y.cpu(), torch.from_numpy(y32).to(torch.bfloat16))
        assert np.all(np.abs(host(y.float()) - y64) <= (UB + 4 * U) * np.abs(y64))
    else:
        assert y is None
    if quant == "int8":
        q, s = front.int8_rows(y32)
        assert np.array_equal(host(scales), s) and np.array_equal(host(codes), q)
        assert np.all(np.abs(host(codes) * s[:, None].astype(np.float64) - y64) <= s[:, None] * (0.5 + 127 * 8 * U))
    elif quant != "none":
        b = y32.reshape(T, H // 128, 128)
        a = np.abs(b).max(2)
        s = np.where(a > 0, a / np.float32(448), np.float32(1))
        if quant == "fp8_pow2":
            s = np.where(a > 0, np.exp2(np.ceil(np.log2(s.astype(np.float64)))), 1).astype(np.float32)
        assert np.array_equal(host(scales), s)
        q = torch.from_numpy(b / s[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(T, H)
        assert torch.equal(codes.cpu().view(torch.uint8), q.view(torch.uint8))
        v = host(codes.float()) * np.repeat(s, 128, axis=1).astype(np.float64)
        assert np.all(np.abs(v - y64) <= (2.0 ** -4 + 8 * U) * np.abs(y64) + np.repeat(s, 128, axis=1) * 2.0 ** -10)


def test_fp8_codes_are_the_dispatch_quantisers_for_bf16_values():
    """A weight and rows that leave y exactly bf16: the norm's FP8 rows are the
    row quantiser's, in both scale formats."""
    T, H = 9, 1024
    rng = np.random.default_rng(2)
    x = torch.from_numpy(rng.choice([-1.0, 1.0], (T, H)).astype(np.float32)).to(torch.bfloat16).cuda()
    w = torch.from_numpy(rng.normal(size=H).astype(np.float32)).to(torch.bfloat16).cuda()
    for quant in ("fp8", "fp8_pow2"):
        # mean square 1: eps 2^-60 vanishes, 1/sqrt is exactly 1 and y = x * w
        _, y, c, s = ep.Buffer.add_rmsnorm(x, None, w, 2.0 ** -60, quant)
        c2, s2 = ep.Buffer.quantize_fp8(y, pow2=quant == "fp8_pow2")
        assert torch.equal(y, x * w)
        assert torch.equal(c.view(torch.uint8), c2.view(torch.uint8)) and torch.equal(s, s2)


def test_in_place_stream():
    """The sum may replace the residual, and y the input."""
    rng = np.random.default_rng(3)
    x, r = _rows(rng, 50, 2048, torch.bfloat16), _rows(rng, 50, 2048, torch.bfloat16)
    w = torch.ones(2048, device="cuda")
    hidden, y, c, s = ep.Buffer.add_rmsnorm(x, r, w, EPS, "int8")
    x2, r2, c2, s2 = x.clone(), r.clone(), torch.empty_like(c), torch.empty_like(s)
    ep.ep_add_rmsnorm(x2, r2, w, r2, x2, c2, s2, EPS, "int8")
    assert torch.equal(r2, hidden) and torch.equal(x2, y) and torch.equal(c2, c) and torch.equal(s2, s)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_rows_that_are_not_finite_show(bad):
    rng = np.random.default_rng(4)
    x = _rows(rng, 4, 512, torch.bfloat16)
    x[1, 300] = bad
    w = torch.ones(512, device="cuda")
    _, y, c, s = ep.Buffer.add_rmsnorm(x, None, w, EPS, "int8")
    _, _, cf, sf = ep.Buffer.add_rmsnorm(x, None, w, EPS, "fp8")
    assert torch.isnan(s[1]) and not c[1].any() and torch.isfinite(s[[0, 2, 3]]).all()
    assert torch.isnan(sf[1, 300 // 128]) and torch.isfinite(sf[[0, 2, 3]]).all()
    assert not torch.isfinite(y[1].float()).all() and torch.isfinite(y[[0, 2, 3]].float()).all()
    qc, qs = ep.Buffer.quantize_int8(x)
    assert torch.isnan(qs[1]) and not qc[1].any() and torch.isfinite(qs[[0, 2, 3]]).all()


def test_no_rows():
    x = torch.empty(0, 256, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(256, device="cuda")
    ep.Buffer.add_rmsnorm(x, x, w, EPS, "int8")
    grad, gw = ep.Buffer.add_rmsnorm_bwd(x, w, x)
    assert grad.shape == x.shape and not gw.any()


@pytest.mark.parametrize("T,H", SHAPES + [(513, 2048), (1029, 264), (4300, 64), (1100, 1024),
                                            (2600, 512), (300, 16384)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("joined", [True, False])
def test_add_rmsnorm_bwd(T, H, dtype, joined):
    rng = np.random.default_rng(T + H)
    h, gy = _rows(rng, T, H, dtype), _rows(rng, T, H, torch.bfloat16)
    gh = _rows(rng, T, H, dtype) if joined else None
    w = torch.from_numpy((1 + 0.3 * rng.normal(size=H)).astype(np.float32)).cuda()
    if T % 2:
        w = w.to(torch.bfloat16)
    grad, gw = ep.Buffer.add_rmsnorm_bwd(h, w, gy, gh, EPS)
    again, gw2 = ep.Buffer.add_rmsnorm_bwd(h, w, gy, gh, EPS)
    assert torch.equal(grad, again) and torch.equal(gw, gw2)
    hn, wn, gn = host(h.float()).astype(np.float64), host(w.float()).astype(np.float64), host(gy.float()).astype(np.float64)
    ref, rw = front.rmsnorm_bwd(hn, wn, gn, None if gh is None else host(gh.float()), EPS)
    r = 1 / np.sqrt((hn * hn).mean(1, keepdims=True) + EPS)
    g, n = gn * wn, hn * r
    # terms of the difference: g*w, n*mean, their difference, r, the joined gradient: at most
    # 8 roundings of each magnitude.  The mean adds H products g*w*h whose first one is rounded:
    # sum_i (1 + d_i) a_i with |d_i| <= U is off by up to U sum |a_i|, however much of the sum cancels
    mag = r * (np.abs(g) + np.abs(n) * np.abs(g * n).mean(1, keepdims=True))
    if gh is not None:
        mag = mag + np.abs(host(gh.float()))
    own = UB if dtype == torch.bfloat16 else U
    assert np.all(np.abs(host(grad.float()) - ref) <= 8 * U * mag + own * np.abs(ref) + 1e-37)
    # a column: rstd and n are rounded, and an fp32 sum of p products in a thread rounds p times;
    # then fp64, rounded to the workgroup's partial (where rows share one) and to the result:
    # p + 4.  p = ceil(T / 512 / rows sharing a workgroup), or 2 without sharing's rounding
    # where that is 1: at most ceil(T / 512) + 4 either way
    assert np.all(np.abs(host(gw) - rw) <= (4 + -(-T // 512)) * U * np.abs(gn * n).sum(0) + 1e-37)


def test_bwd_without_weight_gradient_and_in_place():
    rng = np.random.default_rng(8)
    h, gy, gh = (_rows(rng, 77, 1024, torch.bfloat16) for _ in range(3))
    w = torch.ones(1024, device="cuda")
    grad, _ = ep.Buffer.add_rmsnorm_bwd(h, w, gy, gh)
    ep.ep_add_rmsnorm_bwd(h, w, gy, gh, gh, None, None)
    assert torch.equal(grad, gh)


@pytest.mark.parametrize("raw", [False, True])
def test_bwd_workspace_belongs_to_the_call_stream(raw):
    """The workspace a call makes for itself on another stream is not handed
    to the current stream while the call still waits to run."""
    rng = np.random.default_rng(9)
    T, H = 512, 1024
    h, gy = (_rows(rng, T, H, torch.bfloat16) for _ in range(2))
    w = torch.ones(H, device="cuda")
    want = ep.Buffer.add_rmsnorm_bwd(h, w, gy)
    n = ep.ep_add_rmsnorm_bwd_workspace_bytes(T, H) // 4
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
    got = ep.Buffer.add_rmsnorm_bwd(h, w, gy, stream=side.cuda_stream if raw else side)
    mine = torch.full((n,), 7.0, device="cuda")
    torch.cuda.synchronize()
    assert torch.equal(mine, torch.full_like(mine, 7.0))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
