"""The front of an MoE layer as it is used: norm -> scored routing -> plan ->
INT8 (or FP8) dispatch -> expert FFN -> combine, eager, on another stream,
recorded (prepare) and captured into a graph that is replayed on new inputs;
and the training step's backward of the norm and the router."""

from __future__ import annotations

import numpy as np
import pytest
import torch

import combine_ep_plan_amd as ep
from oracle import front
from tests.gpu_util import dev_f32, host

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    ep.load_library()


class Layer:
    """Buffers and weights of one layer for T tokens; run() makes its calls."""

    def __init__(self, T, H, E, k, F, layout, cap=0, R=1, S=0, quant="int8", seed=0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        rn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        self.T, self.H, self.E, self.k, self.F, self.quant, self.gen = T, H, E, k, F, quant, g
        self.x, self.r = rn(T, H).to(torch.bfloat16), rn(T, H).to(torch.bfloat16)
        self.nw = (1 + 0.1 * rn(H)).to(torch.bfloat16)
        self.router, self.bias = rn(H, E) / H ** 0.5, 0.05 * rn(E)
        self.rule = ep.RouteRule("sigmoid", 4, 2, "top2", True, 2.0)
        self.group = ep.Group(E, R, H, k, T, layout, capacity=cap, slots_per_rank=S,
                              slot_mode="inference" if layout == "static" else "training")
        self.h = ep.Handle(self.group, T)
        self.w1 = ep.Buffer.quantize_int8((rn(E, 2 * F, H) / H ** 0.5).to(torch.bfloat16))
        self.w2 = ep.Buffer.quantize_int8((rn(E, H, F) / F ** 0.5).to(torch.bfloat16))
        rows = self.h.recv_rows
        e = lambda *s, d=torch.bfloat16: torch.zeros(*s, dtype=d, device="cuda")  # noqa: E731
        self.hid, self.y = e(T, H), e(T, H)
        self.q, self.qs = e(T, H, d=torch.int8), e(T, d=torch.float32)
        self.logits = e(T, E, d=torch.float32)
        self.idx, self.w = e(T, k, d=torch.int32), e(T, k, d=torch.float32)
        self.recv, self.rs = e(rows, H, d=torch.int8), e(rows, d=torch.float32)
        self.act, self.out = e(rows, F), e(rows, H)
        self.aq, self.as_ = e(rows, F, d=torch.int8), e(rows, d=torch.float32)
        self.z = e(T, H)

    def norm(self, stream=None):
        ep.ep_add_rmsnorm(self.x, self.r, self.nw, self.hid, self.y, self.q, self.qs, 1e-6, self.quant, stream)

    def gate(self):
        torch.mm(self.y.float(), self.router, out=self.logits)

    def experts(self, stream=None):
        h = self.h.ptr
        ep.ep_route_scored(h, self.rule, self.logits, self.bias, self.idx, self.w, None, stream)
        ep.ep_plan(h, self.idx, stream)
        ep.ep_dispatch_quantized(h, self.q, self.qs, None, self.recv, self.rs, None, None, stream)
        ep.ep_expert_gemm_int8_swiglu(h, self.recv, self.rs, *self.w1, None, None, self.act, stream)
        ep.ep_quantize_int8(self.act, self.aq, self.as_, stream)
        ep.ep_expert_gemm_int8(h, self.aq, self.as_, *self.w2, None, None, self.out, stream)
        ep.ep_combine(h, self.out, self.w, self.z, stream)

    def run(self):
        self.norm()
        self.gate()
        self.experts()

    def outputs(self):
        return [t.clone() for t in (self.hid, self.y, self.q, self.qs, self.idx, self.w, self.z)]

    def renew(self, seed):
        self.gen.manual_seed(seed)
        for t in (self.x, self.r):
            t.copy_(torch.randn(t.shape, generator=self.gen, device="cuda"))


def _reference(L):
    """The layer in 64 bits from the same inputs, the routing ids given."""
    x, r = host(L.x.float()).astype(np.float64), host(L.r.float()).astype(np.float64)
    hid = host((L.x.float() + L.r.float()).to(torch.bfloat16).float())
    assert np.array_equal(host(L.hid.float()), hid) and x.shape == r.shape
    y, _ = front.rmsnorm(hid, host(L.nw.float()), 1e-6)
    ri, rw, _ = front.route_scored(host(L.logits), L.k, "sigmoid", host(L.bias), 4, 2, True, True, 2.0)
    assert np.array_equal(host(L.idx), ri)
    z = np.zeros_like(y)
    w1 = host(L.w1[0]).astype(np.float64) * host(L.w1[1])[..., None]
    w2 = host(L.w2[0]).astype(np.float64) * host(L.w2[1])[..., None]
    for t in range(L.T):
        for j in range(L.k):
            e = ri[t, j]
            if e >= 0:
                a = front.swiglu((w1[e] @ y[t])[None])[0]
                z[t] += rw[t, j] * (w2[e] @ a)
    return z


@pytest.mark.parametrize("layout,cap,R,S", [("ht", 0, 1, 0), ("ll", 24, 1, 0), ("static", 0, 4, 2)])
def test_layer_against_64_bits(layout, cap, R, S):
    """Two INT8 roundings of rows (each value off by up to half of amax / 127:
    for bell-shaped rows about 0.9% of their rms) and bf16 ones of results: the
    layer is within 3% of the exact one, norm-wise."""
    L = Layer(24, 256, 16, 4, 192, layout, cap, R, S)
    L.run()
    z = _reference(L)
    got = host(L.z.float()).astype(np.float64)
    assert np.linalg.norm(got - z) <= 0.03 * np.linalg.norm(z)
    assert L.h.status() == 0


@pytest.mark.parametrize("layout,T", [("ht", 24), ("ht", 700), ("ll", 24), ("static", 300)])
def test_streams_recorded_calls_and_graphs_agree(layout, T):
    L = Layer(T, 256, 16, 4, 192, layout, cap=T, R=4 if layout == "static" else 1, S=2)
    L.run()
    want = L.outputs()
    # another stream, ordered behind the current one
    side = torch.cuda.Stream()
    for t in (L.y, L.z, L.q, L.idx, L.w):
        t.zero_()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        L.run()
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(L.outputs(), want))
    # recorded calls
    first, rest = ep.prepare(L.norm), ep.prepare(L.experts)
    for t in (L.y, L.z, L.q, L.idx, L.w):
        t.zero_()
    first()
    L.gate()
    rest()
    assert all(torch.equal(a, b) for a, b in zip(L.outputs(), want))
    # a captured graph, replayed on new inputs with eager work in between
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        L.norm()
        L.experts()
    for seed in (1, 2, 3):
        L.renew(seed)
        L.run()
        want = L.outputs()
        for t in (L.y, L.z, L.q, L.idx, L.w):
            t.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(L.outputs(), want)), seed


def test_fp8_rows_of_the_norm_feed_the_fp8_product():
    """quant="fp8": the norm's rows dispatched as they are and multiplied by
    the FP8 GEMM are what the bf16 y, quantised by the FP8 dispatch, gives up
    to the rounding of y to bf16 (2^-8) in front of that quantiser."""
    T, H, E, k, N = 64, 256, 8, 2, 128
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    x = torch.randn(T, H, generator=g, device="cuda").to(torch.bfloat16)
    w = torch.ones(H, device="cuda")
    group = ep.Group(E, 1, H, k, T, "ht")
    b, h = ep.Buffer(group), ep.Handle(group, T)
    idx, tw = h.route_scored(torch.randn(T, E, generator=g, device="cuda"), ep.RouteRule())
    h.plan(idx)
    we, se = b.quantize_fp8(torch.randn(E, N, H, generator=g, device="cuda").to(torch.bfloat16))
    _, y, c, s = b.add_rmsnorm(x, None, w, quant="fp8")
    (rc, rs), _, rw, _, _ = b.dispatch_quantized(c, s, tw, h)
    one = b.expert_gemm_fp8(rc, rs, we, se, h)
    (r2, s2), _, rw2, _, _ = b.dispatch(y, idx, tw, handle=h, fp8=True)
    two = b.expert_gemm_fp8(r2, s2, we, se, h)
    assert torch.equal(rw, rw2)
    a, d = host(one.float()).astype(np.float64), host(two.float()).astype(np.float64)
    # both within e4m3's half step (2^-4 of each value, about 0.36 of it rms) of the exact product
    assert np.linalg.norm(a - d) <= 2 * 2.0 ** -4 * np.linalg.norm(d)


def test_training_backward_of_the_front():
    """Loss = <gz, y> + <gh, hidden> + <gw, weights>: the norm's and router's
    backward calls, through the router's weights, against the 64-bit chain."""
    T, H, E, k = 40, 128, 16, 4
    rng = np.random.default_rng(9)
    x, r = (torch.from_numpy(rng.normal(size=(T, H)).astype(np.float32)).to(torch.bfloat16).cuda() for _ in range(2))
    nw, W = dev_f32(1 + 0.1 * rng.normal(size=H)), dev_f32(rng.normal(size=(H, E)) / H ** 0.5)
    gw = dev_f32(rng.normal(size=(T, k)))
    gh = torch.from_numpy(rng.normal(size=(T, H)).astype(np.float32)).to(torch.bfloat16).cuda()
    hid, y, _, _ = ep.Buffer.add_rmsnorm(x, r, nw)
    logits = y.float() @ W
    h = ep.Handle(ep.Group(E, 1, H, k, T, "ht"), T)
    rule = ep.RouteRule("softmax", renormalise=False)
    idx, w, s = h.route_scored(logits, rule, scores=True)
    gl = h.route_scored_bwd(logits, rule, idx, gw)
    gy = (gl @ W.t()).to(torch.bfloat16)
    grad, gnw = ep.Buffer.add_rmsnorm_bwd(hid, nw, gy, gh)
    ref_l, _ = front.route_scored_bwd(host(logits), host(idx), host(gw), None, "softmax", False, 1.0)
    gx, gn = front.rmsnorm_bwd(host(hid.float()), host(nw), ref_l @ host(W).astype(np.float64).T,
                               host(gh.float()), 1e-6)
    # bf16 roundings of gy and of the result, each 2^-8 of its value at most
    assert np.linalg.norm(host(grad.float()) - gx) <= 2 * 2.0 ** -8 * np.linalg.norm(gx)
    assert np.linalg.norm(host(gnw) - gn) <= 2 * 2.0 ** -8 * np.linalg.norm(gn)
