"""FP8 rows of the norm whose blocks are so small that amax / 448 is below the
smallest normal float: still the FP8 row quantiser's codes and scales."""

from __future__ import annotations

import numpy as np
import pytest
import torch

import combine_ep_plan_amd as ep
from tests.gpu_util import host

pytestmark = pytest.mark.gpu
F = np.float32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    ep.load_library()


def _signs(rng, T, H):
    return torch.from_numpy(rng.choice([F(-1), F(1)], (T, H))).to(torch.bfloat16).cuda()


@pytest.mark.parametrize("T", [5, 4099])
@pytest.mark.parametrize("quant", ["fp8", "fp8_pow2"])
def test_tiny_blocks_quantise_like_the_dispatch(T, quant):
    """Rows of 1 and -1 and eps = 2^-60: y is the bf16 weight.  Block i's largest
    value is near 2^(-114 - i), down to bf16's smallest."""
    blocks = 20
    H = 128 * blocks
    rng = np.random.default_rng(T)
    w = np.ldexp(rng.random((blocks, 128)) + 0.5, -114 - np.arange(blocks)[:, None]).astype(F).reshape(-1)
    wt = torch.from_numpy(w).to(torch.bfloat16).cuda()
    x = _signs(rng, T, H)
    _, y, codes, scales = ep.Buffer.add_rmsnorm(x, None, wt, 2.0 ** -60, quant)
    assert torch.equal(y.view(torch.int16), (x * wt).view(torch.int16))
    c2, s2 = ep.Buffer.quantize_fp8(y, pow2=quant == "fp8_pow2")
    assert torch.equal(scales, s2) and torch.equal(codes.view(torch.uint8), c2.view(torch.uint8))
    assert (host(scales)[0] < 2.0 ** -126).any() == (quant == "fp8")


def test_blocks_whose_scale_would_round_to_zero():
    """fp32 values below 448 * 2^-150: the scale stays the smallest float, so
    the codes are the values over it and no quotient is infinite."""
    H = 256
    steps = np.arange(H) % 200 - 100                 # y in steps of 2^-149, |y| <= 100 steps
    w = np.ldexp(steps.astype(np.float64), -149).astype(F)
    x = _signs(np.random.default_rng(1), 3, H)
    _, _, codes, scales = ep.Buffer.add_rmsnorm(x, None, torch.from_numpy(w).cuda(), 2.0 ** -60, "fp8", y=False)
    assert np.all(host(scales) == F(2.0 ** -149))
    want = (x.float() * torch.from_numpy(steps.astype(F)).cuda()).to(torch.float8_e4m3fn).float()
    assert torch.equal(codes.float(), want)
