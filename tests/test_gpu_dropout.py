"""GPU parity of dropout: the mask bit for bit, kept values to the rounding of
their type, the backward as the same call."""

from __future__ import annotations

import numpy as np
import pytest
import torch

import combine_ep_plan_amd as ep
from oracle import dense
from tests.gpu_util import host

pytestmark = pytest.mark.gpu
SEED, OFFSET = 0x9ABCDEF012345678, 0x1_0000_0005


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    ep.load_library()


def _want(x, r, p, dtype, seed=SEED, offset=OFFSET):
    """The formula in float64, rounded to fp32 and then to the type: products of 24-bit numbers are
    exact in float64, so with bf16 x the sum is too unless the exponents lie 20 bits apart, and its
    fp32 rounding is the fma's."""
    f = dense.dropout_factor(tuple(x.shape), p, seed, offset)
    v = np.where(f > 0, host(x.double()) * f, 0.0)
    if r is not None:
        v = v + host(r.double())
    return torch.from_numpy(v).float().to(dtype)


@pytest.mark.parametrize("shape", [(1, 8), (3, 24), (5, 1000), (2, 3, 64), (130, 4096)])
@pytest.mark.parametrize("xt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("ot", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("residual", [False, True])
def test_dropout(shape, xt, ot, residual):
    g = torch.Generator().manual_seed(sum(shape))
    x = torch.randn(shape, generator=g).to(xt).cuda()
    r = torch.randn(shape, generator=g).to(ot).cuda() if residual else None
    rng = ep.rng_state(SEED, OFFSET)
    for p in (0.1, 0.5):
        y = ep.Buffer.dropout(x, p, rng, r, ot)
        assert y.dtype == ot
        want = _want(x, r, p, ot)
        if xt == torch.bfloat16:
            assert torch.equal(y.cpu(), want)
        else:   # the sum of an fp32 product may round twice in float64: half a step of fp32 more
            e = 2.0 ** -24 * (want.abs() + (0 if r is None else r.cpu().float().abs()))
            step = 0 if ot == torch.float32 else 2.0 ** -7 * want.float().abs()   # a bf16 neighbour across a tie
            assert torch.all((y.cpu().double() - want.double()).abs() <= 2 * e + step)
            assert (y.cpu() == want).float().mean() > 0.999


@pytest.mark.parametrize("p,kept", [(0.0, 65536), (1.0, 0), (1e-9, 65536), (1 - 1e-9, 0), (2.0 ** -16, 65535)])
def test_probabilities_at_the_ends(p, kept):
    x = torch.randn(40, 512).to(torch.bfloat16).cuda()
    y = ep.Buffer.dropout(x, p, ep.rng_state(3, 4))
    if kept == 65536:
        assert torch.equal(y, x)
    elif kept == 0:
        assert torch.count_nonzero(y) == 0
    else:
        assert torch.equal(y.cpu(), _want(x, None, p, torch.bfloat16, 3, 4))


def test_dropped_values_do_not_count_whatever_they_are():
    x = torch.full((16, 256), float("nan"), device="cuda", dtype=torch.bfloat16)
    x[::2] = float("inf")
    r = torch.randn(16, 256, device="cuda")
    y = ep.Buffer.dropout(x, 0.5, ep.rng_state(1, 2), r)
    f = torch.from_numpy(dense.dropout_factor((16, 256), 0.5, 1, 2)).cuda()
    assert torch.equal(y[f == 0], r[f == 0]) and not torch.isfinite(y[f > 0]).any()


def test_the_backward_is_the_same_mask():
    x, p = torch.ones(64, 320, device="cuda"), 0.3
    rng = ep.rng_state(11, 12)
    y, g = ep.Buffer.dropout(x, p, rng), ep.Buffer.dropout(x * 2, p, rng)
    assert torch.equal(g, y * 2)
    # differences of the output by the input, one value at a time
    d = ep.Buffer.dropout(x + 1, p, rng) - y
    assert torch.equal(d, y)


def test_offsets_and_seeds_give_other_masks():
    x = torch.ones(256, 256, device="cuda", dtype=torch.bfloat16)
    masks = [ep.Buffer.dropout(x, 0.5, ep.rng_state(s, o)) != 0 for s, o in
             ((1, 0), (1, 1), (2, 0), (1, 1 << 32), (1 + (1 << 32), 0))]
    n = x.numel()
    for i, a in enumerate(masks):
        assert abs(a.float().mean().item() - 0.5) < 6 * 0.5 / n ** 0.5
        for b in masks[:i]:   # equal where both stay or both go: half of the places
            assert abs((a == b).float().mean().item() - 0.5) < 6 * 0.5 / n ** 0.5


def test_counters_past_32_bits_of_values():
    """More than 2^32 values: the block index is 64 bits wide where it is used (2^29 blocks here; the
    last rows against the formula)."""
    T, H = (1 << 20) + 3, 4096
    x = torch.ones(T, H, device="cuda", dtype=torch.bfloat16)
    y = ep.Buffer.dropout(x, 0.5, ep.rng_state(5, 6))
    first = (T - 2) * H
    n = 2 * H
    words = []
    for b in range(first // 8, (first + n) // 8, 97):
        words.append((b, dense.philox((b & dense.M32, b >> 32, 6, 0), (5, 0))))
    flat = y.view(-1)
    for b, w in words:
        got = flat[8 * b:8 * b + 8].float().cpu().tolist()
        want = [2.0 if ((w[c // 2] >> (16 * (c % 2))) & 0xFFFF) < 32768 else 0.0 for c in range(8)]
        assert got == want, b


def test_in_place_empty_and_streams():
    x = torch.randn(33, 512, device="cuda").to(torch.bfloat16)
    r = torch.randn(33, 512, device="cuda").to(torch.bfloat16)
    rng = ep.rng_state(7, 8)
    want = ep.Buffer.dropout(x, 0.2, rng, r)
    a, b = r.clone(), x.clone()
    ep.ep_dropout(x, a, a, 0.2, rng)          # into the residual
    ep.ep_dropout(b, r, b, 0.2, rng)          # into x
    assert torch.equal(a, want) and torch.equal(b, want)
    assert ep.Buffer.dropout(x[:0], 0.2, rng).shape == (0, 512)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y = ep.Buffer.dropout(x, 0.2, rng, r, stream=s)
    s.synchronize()
    assert torch.equal(y, want)
    with pytest.raises(ValueError):
        ep.Buffer.dropout(x.t(), 0.2, rng)
    with pytest.raises(ep.EpError):
        ep.Buffer.dropout(x, 1.5, rng)


def test_replays_read_the_state_anew():
    x = torch.randn(64, 1024, device="cuda").to(torch.bfloat16)
    rng, out = ep.rng_state(1, 0), torch.empty(64, 1024, device="cuda", dtype=torch.bfloat16)
    ep.ep_dropout(x, None, out, 0.5, rng)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ep.ep_dropout(x, None, out, 0.5, rng)
    step = ep.prepare(lambda: ep.ep_dropout(x, None, out, 0.5, rng))
    for i in range(4):
        rng.copy_(ep.rng_state(1, i))
        want = ep.Buffer.dropout(x, 0.5, ep.rng_state(1, i))
        graph.replay()
        assert torch.equal(out, want)
        out.zero_()
        step()
        assert torch.equal(out, want)
