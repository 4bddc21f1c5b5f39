"""GPU tests of the layer norm on rows whose values lie further apart than fp32 reaches:
finite rows have finite results, forward and backward.

A row of -M with a few +M, M near the type's largest: h - mean is up to 2 M, beyond
fp32, its standard deviation M / 16 and less, whose reciprocal is a normal fp32 number.
The bounds are test_gpu_layernorm's, with n by its definition in 64 bits."""

from __future__ import annotations

import numpy as np
import pytest
import torch

import combine_ep_plan_amd as ep
from oracle import dense
from tests.gpu_util import host
from tests.test_gpu_layernorm import EPS, U, UB, _check_y, _gpu  # noqa: F401  (_gpu: fixture)

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32

# a row to a workgroup with one, two and four vectors a thread, a row to a wave
SHAPES = [(3, 2048), (600, 8192), (3, 8200), (3, 16392), (4100, 1024), (4097, 2048)]


def _far(T, H, dtype):
    """-M with one +M a row, at another place in each (in the first row the first value)."""
    top = float(torch.finfo(dtype).max)
    h = torch.full((T, H), -top, dtype=dtype)
    h[torch.arange(T), (torch.arange(T) * 37) % H] = top
    h[1] = -h[1]
    return h.cuda()


@pytest.mark.parametrize("T,H", SHAPES)
@pytest.mark.parametrize("stream", [None, BF, F32])
def test_forward(T, H, stream):
    h = _far(T, H, stream or BF)
    x = h if stream is None else torch.zeros(T, H, dtype=BF, device="cuda")
    rng = np.random.default_rng(H)
    w, b = (torch.from_numpy(rng.normal(size=H).astype(np.float32)).cuda() for _ in range(2))
    hidden, y, _, s = ep.Buffer.add_layernorm(x, None if stream is None else h, w, b, EPS, "int8")
    assert torch.equal(hidden, h)
    y64, n, _ = dense.layernorm(host(h.double()), host(w.double()), host(b.double()), EPS)
    assert np.abs(n).max() > np.sqrt(H) - 1
    _check_y(y, y64, n * host(w.double()))
    assert torch.isfinite(s).all()


@pytest.mark.parametrize("T,H", SHAPES + [(3, 64), (300, 2560)])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("p", [0.0, 0.5])
def test_backward(T, H, dtype, p):
    """The stream's gradient is r g, far below the smallest number: joined with one of its own it is that;
    the sums are of grad_y n and grad_y."""
    h = _far(T, H, dtype)
    rng = np.random.default_rng(H)
    gy = torch.from_numpy(rng.normal(size=(T, H)).astype(np.float32)).to(BF).cuda()
    w = torch.from_numpy((1 + 0.3 * rng.normal(size=H)).astype(np.float32)).cuda()
    gh = torch.from_numpy(rng.normal(size=(T, H)).astype(np.float32)).to(dtype).cuda()
    state = ep.rng_state(5, 6) if p else None
    grad, gx, gw, gb = ep.Buffer.add_layernorm_bwd(h, w, gy, gh, EPS, p, state)
    assert torch.equal(grad, gh)
    f = dense.dropout_factor((T, H), p, 5, 6)
    assert torch.equal(gx.cpu(), torch.from_numpy(host(gh.double()) * f).to(gx.dtype))
    _, n, _ = dense.layernorm(host(h.double()), np.ones(H), None, EPS)
    gyn = host(gy.double())
    steps = T / 256 + 2 + 8
    assert np.all(np.abs(host(gw) - (gyn * n).sum(0)) <= steps * U * np.abs(gyn * n).sum(0) + 1e-30)
    assert np.all(np.abs(host(gb) - gyn.sum(0)) <= steps * U * np.abs(gyn).sum(0) + 1e-30)
