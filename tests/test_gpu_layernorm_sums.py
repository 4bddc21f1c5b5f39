"""GPU tests of the layer norm's weight and bias gradients over many rows: training shapes,
and the longest running sums.

Terms of one sign, so that the running sums grow and every rounding counts.  A workgroup
adds the rows it takes in fp32, `passes` of them at most: each addition within half a step
(U) of the sum of the magnitudes, the term itself within 6 (n from its roundings, the
product), a workgroup's rows side by side joined in fp64 and rounded, then fp64 and one
rounding.  The bound of include/ep.h: T / 256 + 2 rows, T / 512 + 2 up to 4096 channels."""

from __future__ import annotations

import pytest
import torch

import combine_ep_plan_amd as ep
from tests.test_gpu_layernorm import EPS, U, _gpu  # noqa: F401  (_gpu: fixture)

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


# rows a thread adds: 16 (eight of 64 channels side by side in a workgroup), 32, 59 (fp32: two side by side), 98, 118,
# 16 (two side by side), 79 (fp32: two), 24 and 20 (two and four vectors a thread), 257
@pytest.mark.parametrize("T,H,dtype", [(65536, 64, BF), (16384, 4096, BF), (30001, 4096, F32), (25000, 7168, F32), (30000, 7168, BF),
                                       (16384, 2048, BF), (40000, 2560, F32), (6001, 12288, BF), (5000, 20480, F32), (131085, 3000, BF)])
def test_sums_of_many_rows(T, H, dtype):
    p = 0.25 if T % 2 == 0 else 0.0
    g = torch.Generator(device="cuda").manual_seed(T + H)
    sign = torch.where(torch.arange(H, device="cuda") % 2 == 0, 4.0, -4.0)   # channels apart: n keeps its sign
    h = torch.empty(T, H, dtype=dtype, device="cuda")
    gy = torch.empty(T, H, dtype=BF, device="cuda")
    gw64, gb64 = (torch.zeros(H, dtype=torch.float64, device="cuda") for _ in range(2))
    parts = range(0, T, 8192)
    for i in parts:
        j = min(i + 8192, T)
        h[i:j] = torch.randn(j - i, H, generator=g, device="cuda") * 0.5 + sign
        gy[i:j] = 0.5 + torch.rand(j - i, H, generator=g, device="cuda")
    w = torch.ones(H, device="cuda")
    state = ep.rng_state(3, 4) if p else None
    _, _, gw, gb = ep.Buffer.add_layernorm_bwd(h, w, gy, None, EPS, p, state)
    for i in parts:
        d, y = h[i:i + 8192].double(), gy[i:i + 8192].double()
        d -= d.mean(1, keepdim=True)
        n = d / torch.sqrt(d.square().mean(1, keepdim=True) + EPS)
        assert torch.all((n > 0).sum(0) * (n < 0).sum(0) < 0.01 * n.shape[0] ** 2)
        gw64 += (y * n).sum(0)
        gb64 += y.sum(0)
    steps = T / (512 if H <= 4096 else 256) + 2 + 8
    # (the few terms of the other sign: a hundredth more of magnitudes)
    assert torch.all((gw.double() - gw64).abs() <= 1.02 * steps * U * gw64.abs())
    assert torch.all((gb.double() - gb64).abs() <= steps * U * gb64)
    again = ep.Buffer.add_layernorm_bwd(h, w, gy, None, EPS, p, state)
    assert torch.equal(gw, again[2]) and torch.equal(gb, again[3])
