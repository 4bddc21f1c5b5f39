"""The dense half of a layer as a program runs it: a training step (layer norm with
dropout and FP8 rows, product, dropout into the stream; backward with data and
weight gradients) and a serving step (shared expert beside the routed experts).
Every step is held against its own 64-bit form on the inputs it was given, and the
whole chain bit for bit against itself on another stream, prepared, and captured."""

from __future__ import annotations

import numpy as np
import pytest
import torch

import combine_ep_plan_amd as ep
from oracle import dense
from tests.gpu_util import host

pytestmark = pytest.mark.gpu
U, UB = 2.0 ** -24, 2.0 ** -8
EPS, P = 1e-5, 0.2


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    ep.load_library()


def _bf16(*shape, std=1.0, seed=0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * std).to(torch.bfloat16).cuda()


class Step:
    """Forward and backward of one sub-layer [T, H] -> [T, H] on fixed buffers."""

    def __init__(self, T, H, pow2, stream_dtype=torch.float32):
        self.T, self.H, self.pow2 = T, H, pow2
        f8 = lambda *s: torch.empty(s, dtype=torch.float8_e4m3fn, device="cuda")  # noqa: E731
        f32 = lambda *s: torch.empty(s, dtype=torch.float32, device="cuda")  # noqa: E731
        bf = lambda *s: torch.empty(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
        Tp, KB = (T + 127) // 128 * 128, H // 128
        self.x, self.res, self.gout = bf(T, H), torch.empty(T, H, dtype=stream_dtype, device="cuda"), bf(T, H)
        self.w, self.b, self.W = bf(H), bf(H), bf(H, H)
        self.rng1, self.rng2 = ep.rng_state(1), ep.rng_state(2)
        self.main = f32(H, H)
        # forward
        self.h, self.y = torch.empty_like(self.res), bf(T, H)
        self.yc, self.ys = f8(T, H), f32(T, KB)
        self.wq = f8(H, H), f32(KB, KB), f8(H, H), f32(KB, KB)
        self.z, self.out = bf(T, H), torch.empty_like(self.res)
        # backward
        self.gz, self.gy = bf(T, H), bf(T, H)
        self.gq = f8(T, H), f32(T, KB), f8(H, Tp), f32(H, Tp // 128)
        self.yt = f8(H, Tp), f32(H, Tp // 128)
        self.gh, self.gx = torch.empty_like(self.res), bf(T, H)
        self.gw, self.gb = f32(H), f32(H)
        self.ws = f32(ep.ep_add_layernorm_bwd_workspace_bytes(T, H) // 4)
        self.gstream = torch.empty_like(self.res)

    def load(self, seed):
        T, H = self.T, self.H
        self.x.copy_(_bf16(T, H, seed=seed))
        self.res.copy_(_bf16(T, H, std=2.0, seed=seed + 1))
        self.gout.copy_(_bf16(T, H, std=0.5, seed=seed + 2))
        self.w.copy_(1 + 0.1 * _bf16(H, seed=seed + 3))
        self.b.copy_(0.1 * _bf16(H, seed=seed + 4))
        self.W.copy_(_bf16(H, H, std=H ** -0.5, seed=seed + 5))
        self.gstream.copy_(_bf16(T, H, seed=seed + 6))
        self.rng1.copy_(ep.rng_state(11, seed))
        self.rng2.copy_(ep.rng_state(12, seed))
        self.main.fill_(1.0)

    def run(self, s=None):
        q = "fp8_pow2" if self.pow2 else "fp8"
        ep.ep_add_layernorm(self.x, self.res, self.w, self.b, self.h, self.y, self.yc, self.ys, EPS, q, P, self.rng1, s)
        ep.ep_quantize_fp8_2d(self.W, *self.wq, block="square", pow2=self.pow2, stream=s)
        ep.ep_linear_fp8(self.yc, self.ys, self.wq[0], self.wq[1], None, self.z, pow2=self.pow2, stream=s)
        ep.ep_dropout(self.z, self.h, self.out, P, self.rng2, s)
        ep.ep_dropout(self.gout, None, self.gz, P, self.rng2, s)
        ep.ep_quantize_fp8_2d(self.gz, *self.gq, block="rows", pow2=self.pow2, stream=s)
        ep.ep_linear_fp8(self.gq[0], self.gq[1], self.wq[2], self.wq[3], None, self.gy, pow2=self.pow2, stream=s)
        ep.ep_quantize_fp8_2d(self.y, None, None, *self.yt, block="rows", pow2=self.pow2, stream=s)
        ep.ep_linear_fp8(self.gq[2], self.gq[3], *self.yt, self.main, self.main, pow2=self.pow2, stream=s)
        ep.ep_add_layernorm_bwd(self.h, self.w, self.gy, self.gstream, self.gh, self.gx, self.gw, self.gb, self.ws, EPS,
                                P, self.rng1, s)

    def results(self):
        return [t.clone() for t in (self.h, self.y, self.z, self.out, self.gz, self.gy, self.main, self.gh, self.gx,
                                    self.gw, self.gb, self.ys, *self.wq[1::2], *self.gq[1::2], self.yt[1])] + \
            [t.view(torch.uint8).clone() for t in (self.yc, *self.wq[::2], *self.gq[::2], self.yt[0])]


def _same(a, b):
    return all(torch.equal(p, q) for p, q in zip(a, b))


def _product(got, x, xs, w, ws, square, add=None):
    """Within the FP8 product's bound (test_gpu_linear_fp8.py), from the operands it was given."""
    from tests.test_gpu_linear_fp8 import _cut
    p = (host(x.view(torch.uint8)), host(xs), host(w.view(torch.uint8)), host(ws))
    want, mag = dense.linear(*p, square, add)
    K = p[0].shape[1]
    tol = (256 + 4 * (K // 128)) * U * mag + (0 if got.dtype == torch.float32 else _cut(p, square))
    own = U if got.dtype == torch.float32 else UB
    assert np.all(np.abs(host(got.double()) - want) <= tol + own * (np.abs(want) + tol) + (0 if add is None else 2 * U * np.abs(add)))


@pytest.mark.parametrize("T,H", [(1, 128), (70, 256), (257, 640)])
@pytest.mark.parametrize("pow2", [False, True])
def test_training_step(T, H, pow2):
    st = Step(T, H, pow2)
    st.load(T + H)
    st.run()
    f1 = dense.dropout_factor((T, H), P, 11, T + H)
    f2 = dense.dropout_factor((T, H), P, 12, T + H)
    h = torch.from_numpy(host(st.x.double()) * f1 + host(st.res.double())).float()
    assert torch.equal(st.h.cpu(), h)
    y64, n64, _ = dense.layernorm(h.numpy(), host(st.w.double()), host(st.b.double()), EPS)
    assert np.all(np.abs(host(st.y.double()) - y64) <= UB * np.abs(y64) + 8 * U * (np.abs(y64) + 1))
    _product(st.z, st.yc, st.ys, st.wq[0], st.wq[1], True)
    out = torch.from_numpy(host(st.z.double()) * f2 + host(st.h.double())).float()
    assert torch.all((st.out.cpu() - out).abs() <= 2 * U * (out.abs() + st.h.cpu().abs()))
    assert torch.equal(st.gz.cpu(), torch.from_numpy(host(st.gout.double()) * f2).float().to(torch.bfloat16))
    _product(st.gy, st.gq[0], st.gq[1], st.wq[2], st.wq[3], True)
    _product(st.main, st.gq[2], st.gq[3], st.yt[0], st.yt[1], False, np.ones((H, H)))
    # the weight gradient's operands are the gradient and the rows, by columns of 128 tokens
    gz, y = np.zeros((H, (T + 127) // 128 * 128), np.float32), np.zeros((H, (T + 127) // 128 * 128), np.float32)
    gz[:, :T], y[:, :T] = host(st.gz.float()).T, host(st.y.float()).T
    for v, (c, s) in ((gz, st.gq[2:]), (y, st.yt)):
        back = dense.fp8_values(host(c.view(torch.uint8)), host(s), 1)
        step = np.repeat(host(s).astype(np.float64), 128, 1)
        assert np.all(np.abs(back - v) <= 2.0 ** -4 * np.abs(v) * (1 + 4 * U) + step * 2.0 ** -10)
    g64, gw64, gb64 = dense.layernorm_bwd(host(st.h.double()), host(st.w.double()), host(st.gy.double()),
                                          host(st.gstream.double()), EPS)
    scale = np.abs(g64).max()
    assert np.all(np.abs(host(st.gh.double()) - g64) <= 64 * U * scale * H ** 0.5)
    assert np.all(np.abs(host(st.gx.double()) - g64 * f1) <= UB * np.abs(g64 * f1) + 64 * U * scale * H ** 0.5)
    gyn = host(st.gy.double())
    assert np.all(np.abs(host(st.gw) - gw64) <= 64 * U * np.abs(gyn * n64).sum(0) + 1e-30)
    assert np.all(np.abs(host(st.gb) - gb64) <= 64 * U * np.abs(gyn).sum(0) + 1e-30)


@pytest.mark.parametrize("pow2", [False, True])
def test_the_step_on_another_stream_prepared_and_captured(pow2):
    st = Step(300, 512, pow2)
    st.load(3)
    st.run()
    want = st.results()
    s = torch.cuda.Stream()
    st.load(3)
    s.wait_stream(torch.cuda.current_stream())
    st.run(s)
    s.synchronize()
    assert _same(want, st.results())
    prepared = ep.prepare(st.run)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        st.run()
    for i in range(3):
        st.load(10 * i)
        st.run()
        want = st.results()
        for run in (graph.replay, prepared):
            st.load(10 * i)
            run()
            assert _same(want, st.results()), i


def test_two_steps_at_once():
    """Two steps of their own buffers on two streams at a time share nothing."""
    steps = [Step(200, 384, False), Step(333, 256, True)]
    want = []
    for k, st in enumerate(steps):
        st.load(k)
        st.run()
        want.append(st.results())
    streams = [torch.cuda.Stream() for _ in steps]
    for _ in range(4):
        for k, (st, s) in enumerate(zip(steps, streams)):
            st.load(k)
            s.wait_stream(torch.cuda.current_stream())
        for _ in range(2):   # the second run adds to the main gradient again: only the rest is compared
            for st, s in zip(steps, streams):
                st.run(s)
        torch.cuda.synchronize()
        for st, w in zip(steps, want):
            got = st.results()
            assert _same(got[:6] + got[7:], w[:6] + w[7:])


@pytest.mark.parametrize("T", [1, 5, 48, 130])
def test_shared_expert_beside_the_routed_ones(T):
    """norm -> shared expert (SwiGLU product, rows to FP8, second product) added to combine's rows."""
    H, I, E, k = 256, 384, 8, 2
    g = ep.Group(E, 1, H, k, T, "ht")
    h, buf = ep.Handle(g, T), ep.Buffer(g)
    x, w = _bf16(T, H, seed=T), torch.ones(H, device="cuda", dtype=torch.bfloat16)
    w1, w2 = _bf16(2 * I, H, std=H ** -0.5, seed=2), _bf16(H, I, std=I ** -0.5, seed=3)
    c1, s1, _, _ = buf.quantize_fp8_2d(w1, "square", transposed=False)
    c2, s2, _, _ = buf.quantize_fp8_2d(w2, "square", transposed=False)
    hidden, y, yc, ys = buf.add_layernorm(x, None, w, None, EPS, "fp8")
    idx, tw = h.route(torch.randn(T, E, generator=torch.Generator().manual_seed(T)).cuda())
    recv, _, _, h, _ = buf.dispatch(y, idx, tw, handle=h.plan(idx))
    routed = buf.combine(recv, h, tw)               # experts that return their rows
    act = buf.linear_fp8(yc, ys, c1, s1, swiglu=True)
    ac, asc = buf.quantize_fp8(act)
    out = buf.linear_fp8(ac, asc, c2, s2, addend=routed)
    assert act.shape == (T, I) and out.shape == (T, H) and out.dtype == torch.bfloat16
    _product(out, ac, asc, c2, s2, True, host(routed.double()))
    gate_up, mag = dense.linear(host(yc.view(torch.uint8)), host(ys), host(c1.view(torch.uint8)), host(s1), True)
    want = gate_up[:, 0::2] / (1 + np.exp(-gate_up[:, 0::2])) * gate_up[:, 1::2]
    size = mag[:, 0::2] * (1 + np.abs(gate_up[:, 1::2])) + mag[:, 1::2] * (1 + np.abs(gate_up[:, 0::2]))
    # what the matrix cores cut is at most 8 * 2^-12 of each group's largest products, so 2^-9 of the terms
    assert np.all(np.abs(host(act.double()) - want) <= UB * np.abs(want) + 2.0 ** -9 * size)
