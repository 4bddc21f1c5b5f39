"""GPU parity of the residual layer norm with dropout, its 8-bit outputs and its
backward.

The stream h is exact (one fma, one rounding).  y = fma(n, w, b) with n from two
roundings and the once-rounded 1/sqrt: |n| off by 3 half steps, so y by
3 U |n w| + U |y| before its own type's rounding (U = 2^-24); the sums run in
float64.  FP8 values add half a step of e4m3, INT8 half a step of the scale."""

from __future__ import annotations

import numpy as np
import pytest
import torch

import combine_ep_plan_amd as ep
from oracle import dense
from tests.gpu_util import host

pytestmark = pytest.mark.gpu
U, UB = 2.0 ** -24, 2.0 ** -8
EPS = 1e-5
SEED, OFFSET = 77, 5


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    ep.load_library()


def _rows(rng, T, H, dtype, std=1.0):
    x = rng.normal(size=(T, H)) * std * np.exp(rng.normal(size=H) * 0.5) + rng.normal(size=H)
    return torch.from_numpy(x.astype(np.float32)).to(dtype).cuda()


def _joined(x, r, p):
    f = dense.dropout_factor(tuple(x.shape), p, SEED, OFFSET)
    v = host(x.double()) * f
    if r is not None:
        v = v + host(r.double())
    return torch.from_numpy(v).float().to(torch.bfloat16 if r is None else r.dtype)


SHAPES = [(1, 8), (3, 128), (2, 512), (5, 520), (4, 1024), (1, 7168), (130, 256), (33, 4096), (2, 8192),
          (2, 8200), (3, 16384), (2, 32768), (700, 384)]


def _check_y(y, y64, nw64, extra=UB):
    assert np.all(np.abs(host(y.float()) - y64) <= extra * np.abs(y64) + 4 * U * (np.abs(nw64) + np.abs(y64)) + 1e-30)


@pytest.mark.parametrize("T,H", SHAPES)
@pytest.mark.parametrize("residual", [None, torch.bfloat16, torch.float32])
@pytest.mark.parametrize("quant", ["none", "int8", "fp8", "fp8_pow2"])
@pytest.mark.parametrize("p", [0.0, 0.3])
def test_add_layernorm(T, H, residual, quant, p):
    if quant.startswith("fp8") and H % 128:
        H = (H + 127) // 128 * 128 if H < 32768 else H
    rng = np.random.default_rng(T * 31 + H)
    x = _rows(rng, T, H, torch.bfloat16)
    r = None if residual is None else _rows(rng, T, H, residual, 2.0)
    wt = torch.bfloat16 if T % 2 else torch.float32
    w = torch.from_numpy((1 + 0.3 * rng.normal(size=H)).astype(np.float32)).to(wt).cuda()
    b = torch.from_numpy((0.2 * rng.normal(size=H)).astype(np.float32)).to(wt).cuda() if H % 3 else None
    if T > 2:
        x[T // 2] = 0
        if r is not None:
            r[T // 2] = 0
    want_y = quant in ("none", "fp8")
    state = ep.rng_state(SEED, OFFSET) if p else None
    hidden, y, codes, scales = ep.Buffer.add_layernorm(x, r, w, b, EPS, quant, y=want_y, dropout=p, rng=state)
    h_ref = x.cpu() if r is None and not p else _joined(x, r, p)
    assert torch.equal(hidden.cpu(), h_ref)
    wn, bn = host(w.double()), None if b is None else host(b.double())
    y64, n64, _ = dense.layernorm(h_ref.double().numpy(), wn, bn, EPS)
    nw = n64 * wn
    slack = 4 * U * (np.abs(nw) + np.abs(y64))
    if want_y:
        _check_y(y, y64, nw)
    else:
        assert y is None
    if quant == "int8":
        s = host(scales).astype(np.float64)
        a = np.abs(y64).max(1)
        assert np.all(np.abs(s - np.where(a > 0, a / 127, 1)) <= slack.max(1) / 127 + 2 * U * s)
        assert np.all(np.abs(host(codes) * s[:, None] - y64) <= s[:, None] * (0.5 + 128 * 4 * U) + slack)
    elif quant != "none":
        s = host(scales).astype(np.float64)
        a = np.abs(y64).reshape(T, H // 128, 128).max(2)
        sl = slack.reshape(T, H // 128, 128).max(2)
        if quant == "fp8":
            assert np.all(np.abs(s - np.where(a > 0, a / 448, 1)) <= sl / 448 + 2 * U * s)
        else:   # a power of two, the next above amax / 448 unless that lies within the rounding of one
            assert np.all(np.frexp(s)[0] == 0.5)
            near = (a + sl) / 448
            assert np.all((s >= (a - sl) / 448) & ((s < 2 * near) | (a == 0)))
        se = np.repeat(s, 128, axis=1)
        assert np.all(np.abs(host(codes.float()) * se - y64) <= 2.0 ** -4 * np.abs(y64) + se * 2.0 ** -10 + 2 * slack)


@pytest.mark.parametrize("T,H", [(4103, 8), (4096, 512), (4103, 1000), (4097, 2048), (600, 4104)])
@pytest.mark.parametrize("residual", [None, torch.bfloat16, torch.float32])
@pytest.mark.parametrize("quant,p", [("none", 0.0), ("int8", 0.3), ("fp8", 0.3), ("fp8_pow2", 0.0)])
def test_many_rows_a_wave_each(T, H, residual, quant, p):
    test_add_layernorm(T, H, residual, quant, p)


def test_eight_bit_rows_are_the_quantisers_where_y_is_exact_in_bf16():
    """Rows of +-1 in equal number: mean 0, variance 1, n = +-1 up to eps, which 2^-60 hides."""
    T, H = 9, 1024
    rng = np.random.default_rng(2)
    signs = np.stack([rng.permutation(np.repeat([-1.0, 1.0], H // 2)) for _ in range(T)])
    x = torch.from_numpy(signs.astype(np.float32)).to(torch.bfloat16).cuda()
    w = torch.from_numpy(rng.normal(size=H).astype(np.float32)).to(torch.bfloat16).cuda()
    for quant in ("fp8", "fp8_pow2"):
        _, y, c, s = ep.Buffer.add_layernorm(x, None, w, None, 2.0 ** -60, quant)
        c2, s2 = ep.Buffer.quantize_fp8(y, pow2=quant == "fp8_pow2")
        assert torch.equal(y, x * w)
        assert torch.equal(c.view(torch.uint8), c2.view(torch.uint8)) and torch.equal(s, s2)
    _, y, c, s = ep.Buffer.add_layernorm(x, None, w, None, 2.0 ** -60, "int8")
    c2, s2 = ep.Buffer.quantize_int8(y)
    assert torch.equal(c, c2) and torch.equal(s, s2)


def test_large_means_and_constant_rows():
    """A mean of 2^20 standard deviations in an fp32 stream costs nothing; a constant row has variance 0."""
    H = 1000
    rng = np.random.default_rng(5)
    h = (rng.normal(size=(6, H)) + 2.0 ** 20).astype(np.float32)
    h[1], h[2], h[3] = 1e6, -3.0, 0.0
    h[4] = 1e-3 * rng.normal(size=H)
    h[5] *= 1e10
    r = torch.from_numpy(h).cuda()
    x = torch.zeros(6, H, device="cuda", dtype=torch.bfloat16)
    w, b = torch.ones(H, device="cuda"), torch.full((H,), 0.5, device="cuda")
    hidden, y, _, _ = ep.Buffer.add_layernorm(x, r, w, b, EPS)
    assert torch.equal(hidden, r)
    y64, n64, _ = dense.layernorm(h, np.ones(H), np.full(H, 0.5), EPS)
    _check_y(y, y64, n64)
    assert torch.all(y[1:4] == 0.5)
    gy = torch.randn(6, H, device="cuda").to(torch.bfloat16)
    g, _, gw, gb = ep.Buffer.add_layernorm_bwd(r, w, gy, None, EPS)
    g64, gw64, gb64 = dense.layernorm_bwd(h, np.ones(H), host(gy.double()), None, EPS)
    gn = host(gy.double())
    _, n, rs = dense.layernorm(h, np.ones(H), None, EPS)
    A = rs * (np.abs(gn) + np.abs(gn.mean(1, keepdims=True)) + np.abs(n * (gn * n).mean(1, keepdims=True)))
    assert np.all(np.abs(host(g) - g64) <= 12 * U * A)
    assert np.all(np.abs(host(gw) - gw64) <= 12 * U * np.abs(gn * n).sum(0))


def test_rows_that_are_not_finite_are_nan():
    x = torch.randn(4, 256, device="cuda").to(torch.bfloat16)
    x[0, 0], x[1, 77], x[2, 255] = float("inf"), float("nan"), float("-inf")
    w = torch.ones(256, device="cuda")
    _, y, c, s = ep.Buffer.add_layernorm(x, None, w, w, EPS, "fp8")
    assert torch.isnan(y[:3]).all() and torch.isfinite(y[3]).all()
    assert torch.isnan(s[:3]).all() and torch.isfinite(s[3]).all() and torch.all(c[:3].view(torch.uint8) == 0)
    _, _, c, s = ep.Buffer.add_layernorm(x, None, w, w, EPS, "int8", y=False)
    assert torch.isnan(s[:3]).all() and torch.all(c[:3] == 0) and torch.isfinite(s[3])


@pytest.mark.parametrize("T,H", [(3, 512), (5, 7168), (5000, 2048), (4100, 256)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_in_place_stream(T, H, dtype):
    """The sum may replace the residual, and y the branch, while every thread reads the row's first value."""
    rng = np.random.default_rng(3)
    x, r = _rows(rng, T, H, torch.bfloat16), _rows(rng, T, H, dtype, 2.0)
    w = torch.ones(H, device="cuda")
    state = ep.rng_state(1, 2)
    want_h, want_y, _, _ = ep.Buffer.add_layernorm(x, r, w, None, EPS, dropout=0.1, rng=state)
    ep.ep_add_layernorm(x, r, w, None, r, x, eps=EPS, dropout=0.1, rng=state)
    assert torch.equal(r, want_h) and torch.equal(x, want_y)


BWD = [(1, 8), (3, 128), (7, 512), (300, 520), (600, 1000), (130, 1024), (1500, 64), (33, 4096), (520, 2048),
       (2, 8192), (5, 8200), (3, 16384), (2, 32768), (2100, 256), (600, 8200), (270, 16392)]


@pytest.mark.parametrize("T,H", BWD)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("joined", [False, True])
@pytest.mark.parametrize("p", [0.0, 0.4])
def test_backward(T, H, dtype, joined, p):
    """grad: differences of three fp32 terms and their products, each within 10 half steps of the terms'
    magnitudes, then its type's; the sums over rows in fp32 a workgroup's rows at a time (at most
    T / 256 + 2 of them), then in float64."""
    rng = np.random.default_rng(T + H)
    h, gy = _rows(rng, T, H, dtype), torch.from_numpy(rng.normal(size=(T, H)).astype(np.float32)).to(torch.bfloat16).cuda()
    gh = _rows(rng, T, H, dtype) if joined else None
    wt = torch.bfloat16 if T % 2 else torch.float32
    w = torch.from_numpy((1 + 0.3 * rng.normal(size=H)).astype(np.float32)).to(wt).cuda()
    state = ep.rng_state(SEED, OFFSET) if p else None
    grad, gx, gw, gb = ep.Buffer.add_layernorm_bwd(h, w, gy, gh, EPS, p, state)
    assert grad.dtype == dtype and gw.dtype == gb.dtype == torch.float32
    hn, wn, gyn = host(h.double()), host(w.double()), host(gy.double())
    ghn = None if gh is None else host(gh.double())
    g64, gw64, gb64 = dense.layernorm_bwd(hn, wn, gyn, ghn, EPS)
    _, n, r = dense.layernorm(hn, wn, None, EPS)
    g = gyn * wn
    A = r * (np.abs(g) + np.abs(g.mean(1, keepdims=True)) + np.abs(n) * np.abs((g * n).mean(1, keepdims=True)))
    if ghn is not None:
        A = A + np.abs(ghn)
    tol = 10 * U * A
    own = UB if dtype == torch.bfloat16 else U
    assert np.all(np.abs(host(grad.double()) - g64) <= tol + own * (np.abs(g64) + tol))
    if p:
        f = dense.dropout_factor((T, H), p, SEED, OFFSET)
        assert gx.dtype == torch.bfloat16
        assert np.all(np.abs(host(gx.double()) - g64 * f) <= (tol + (UB + U) * (np.abs(g64) + tol)) * f)
    else:
        assert gx is grad
    steps = T / 256 + 2 + 6
    assert np.all(np.abs(host(gw) - gw64) <= steps * U * np.abs(gyn * n).sum(0) + 1e-30)
    assert np.all(np.abs(host(gb) - gb64) <= steps * U * np.abs(gyn).sum(0) + 1e-30)


def test_backward_against_differences():
    """grad_y . y as a function of x, the weight and the bias, by central differences of the forward in
    float64 steps that fp32 holds: eps 0.1 keeps third derivatives small."""
    T, H, d = 2, 16, 2.0 ** -6
    rng = np.random.default_rng(8)
    h = torch.from_numpy(rng.integers(-32, 33, size=(T, H)).astype(np.float32) / 16).cuda()
    w = torch.from_numpy(rng.integers(8, 33, size=H).astype(np.float32) / 16).cuda()
    b = torch.zeros(H, device="cuda")
    gy = torch.from_numpy(rng.integers(-16, 17, size=(T, H)).astype(np.float32) / 8).to(torch.bfloat16).cuda()
    zero = torch.zeros(T, H, device="cuda", dtype=torch.bfloat16)
    grad, _, gw, gb = ep.Buffer.add_layernorm_bwd(h, w, gy, None, 0.1)

    def f(hh, ww, bb):   # from the FP64 form: the kernel's y is bf16, too coarse for differences
        return (dense.layernorm(host(hh), host(ww), host(bb), 0.1)[0] * host(gy.double())).sum()

    _, y, _, _ = ep.Buffer.add_layernorm(zero, h, w, b, 0.1)
    assert np.all(np.abs(host(y.double()) - dense.layernorm(host(h), host(w), host(b), 0.1)[0]) <= 2 * UB * 8)
    for i, j in [(0, 0), (0, 7), (1, 15), (1, 3)]:
        e = torch.zeros_like(h)
        e[i, j] = d
        assert abs((f(h + e, w, b) - f(h - e, w, b)) / (2 * d) - grad[i, j].item()) < 200 * d * d
    for j in (0, 9):
        e = torch.zeros_like(w)
        e[j] = d
        assert abs((f(h, w + e, b) - f(h, w - e, b)) / (2 * d) - gw[j].item()) < 1e-4
        assert abs((f(h, w, b + e) - f(h, w, b - e)) / (2 * d) - gb[j].item()) < 1e-4


def test_backward_outputs_one_at_a_time_empty_and_in_place():
    rng = np.random.default_rng(9)
    T, H = 300, 768
    h, gy = _rows(rng, T, H, torch.bfloat16), _rows(rng, T, H, torch.bfloat16)
    gh, w, state = _rows(rng, T, H, torch.bfloat16), torch.ones(H, device="cuda"), ep.rng_state(1, 1)
    grad, gx, gw, gb = ep.Buffer.add_layernorm_bwd(h, w, gy, gh, EPS, 0.2, state)
    ws = torch.empty(ep.ep_add_layernorm_bwd_workspace_bytes(T, H) // 4, device="cuda")
    one = torch.empty(H, device="cuda")
    ep.ep_add_layernorm_bwd(h, w, gy, gh, None, gx2 := torch.empty_like(gx), None, one, ws, EPS, 0.2, state)
    assert torch.equal(gx2, gx) and torch.equal(one, gb)
    ep.ep_add_layernorm_bwd(h, w, gy, gh, gh, gx2, one, None, ws, EPS, 0.2, state)   # into the stream's gradient
    assert torch.equal(gh, grad) and torch.equal(gx2, gx) and torch.equal(one, gw)
    ep.ep_add_layernorm_bwd(h, w, gy, None, gx2, None, None, None, None, EPS)        # no sums, no workspace
    assert torch.equal(gx2, ep.Buffer.add_layernorm_bwd(h, w, gy, None, EPS)[0])
    g, x, gw, gb = ep.Buffer.add_layernorm_bwd(h[:0], w, gy[:0], None, EPS)
    assert g.shape == (0, H) and torch.count_nonzero(gw) == 0 and torch.count_nonzero(gb) == 0
    hid, y, _, _ = ep.Buffer.add_layernorm(h[:0], gh[:0], w)
    assert hid.shape == y.shape == (0, H)
    with pytest.raises(ep.EpError):
        ep.ep_add_layernorm_bwd(h, w, gy, gh, None, gx2, None, one, ws[:8], EPS, 0.2, state)


def test_streams_prepared_and_captured():
    rng = np.random.default_rng(10)
    T, H = 257, 1024
    x, r = _rows(rng, T, H, torch.bfloat16), _rows(rng, T, H, torch.float32)
    w, b = torch.rand(H, device="cuda"), torch.rand(H, device="cuda")
    gy, state = _rows(rng, T, H, torch.bfloat16), ep.rng_state(3, 0)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    want = ep.Buffer.add_layernorm(x, r, w, b, EPS, "fp8", dropout=0.1, rng=state)
    other = ep.Buffer.add_layernorm(x, r, w, b, EPS, "fp8", dropout=0.1, rng=state, stream=s)
    bwant = ep.Buffer.add_layernorm_bwd(want[0], w, gy, r, EPS, 0.1, state)
    s.wait_stream(torch.cuda.current_stream())
    bother = ep.Buffer.add_layernorm_bwd(want[0], w, gy, r, EPS, 0.1, state, stream=s)
    s.synchronize()
    for p, q in zip(want + bwant, other + bother):
        assert torch.equal(p.view(torch.uint8), q.view(torch.uint8))
    out = [torch.empty_like(t) for t in want]
    bout = [torch.empty_like(t) for t in bwant]
    ws = torch.empty(ep.ep_add_layernorm_bwd_workspace_bytes(T, H) // 4, device="cuda")

    def calls():
        ep.ep_add_layernorm(x, r, w, b, *out, eps=EPS, quant="fp8", dropout=0.1, rng=state)
        ep.ep_add_layernorm_bwd(out[0], w, gy, r, *bout, ws, EPS, 0.1, state)

    step = ep.prepare(calls)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    for i in range(4):
        state.copy_(ep.rng_state(3, i))
        x.copy_(_rows(rng, T, H, torch.bfloat16))
        want = ep.Buffer.add_layernorm(x, r, w, b, EPS, "fp8", dropout=0.1, rng=state)
        bwant = ep.Buffer.add_layernorm_bwd(want[0], w, gy, r, EPS, 0.1, state)
        for run in (graph.replay, step):
            for t in out + bout:
                t.zero_()
            run()
            for p, q in zip(want + bwant, out + bout):
                assert torch.equal(p.view(torch.uint8), q.view(torch.uint8)), i


def test_repeats_bit_for_bit():
    rng = np.random.default_rng(12)
    h, gy = _rows(rng, 3000, 640, torch.bfloat16), _rows(rng, 3000, 640, torch.bfloat16)
    w = torch.ones(640, device="cuda")
    a = ep.Buffer.add_layernorm_bwd(h, w, gy)
    for _ in range(3):
        assert all(torch.equal(p, q) for p, q in zip(a, ep.Buffer.add_layernorm_bwd(h, w, gy)))


def test_offsets_past_32_bits():
    """More than 2^32 values: the last rows as they are alone."""
    T, H = 131090, 32768
    rng = np.random.default_rng(8)
    last = _rows(rng, 3, H, torch.bfloat16)
    gy = _rows(rng, 3, H, torch.bfloat16)
    w, b = torch.ones(H, device="cuda"), torch.ones(H, device="cuda")
    x = torch.zeros(T, H, dtype=torch.bfloat16, device="cuda")
    x[-3:] = last
    _, y, codes, scales = ep.Buffer.add_layernorm(x, None, w, b, EPS, "fp8")
    _, y1, c1, s1 = ep.Buffer.add_layernorm(last, None, w, b, EPS, "fp8")
    assert torch.equal(y[-3:], y1) and torch.equal(scales[-3:], s1)
    assert torch.equal(codes[-3:].view(torch.uint8), c1.view(torch.uint8))
    assert torch.all(y[0] == 1) and torch.all(y[T // 2] == 1)
    y.zero_()
    y[-3:] = gy
    g, _, gw, gb = ep.Buffer.add_layernorm_bwd(x, w, y, None, EPS)
    g1, _, gw1, gb1 = ep.Buffer.add_layernorm_bwd(last, w, gy, None, EPS)
    assert torch.equal(g[-3:], g1) and not g[:-3].any()
    # three rows' terms in another order: two sums, each within half a step
    for a, c in ((gw, gw1), (gb, gb1)):
        assert torch.all((a - c).abs() <= 4 * U * 16 * 8)
