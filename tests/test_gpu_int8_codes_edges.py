"""INT8 codes where the scale is near the smallest normal float: a half of it
is no float there, and a code must still be the integer nearest to the exact
quotient."""

from __future__ import annotations

import numpy as np
import pytest
import torch

import combine_ep_plan_amd as ep
from oracle import front
from tests.gpu_util import host

pytestmark = pytest.mark.gpu
F = np.float32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    ep.load_library()


def _bf16_rows():
    """Rows whose largest value gives a scale in [2^-126, 2^-125), with the
    bf16 values on both sides of every tie (q + 1/2) * scale."""
    rows = []
    for bits in range(0x0380, 0x0480):
        a = np.array([bits << 16], np.uint32).view(F)[0]
        s = F(a * (F(1) / F(127)))
        if not 2.0 ** -126 <= s < 2.0 ** -125:
            continue
        c = ((np.arange(127) + 0.5) * np.float64(s)).astype(F).view(np.uint32) >> 16
        v = np.concatenate([(c << 16).view(F), ((c + 1) << 16).astype(np.uint32).view(F)])
        v = np.where(v <= a, v, F(0))
        rows.append(np.concatenate([[a], v, [-a]]).astype(F))
    return np.stack(rows)


def test_quantize_int8_between_the_smallest_scales():
    x = _bf16_rows()
    x = np.concatenate([x, -x])
    assert x.shape[1] % 8 == 0
    t = torch.from_numpy(x).to(torch.bfloat16)
    assert torch.equal(t.float(), torch.from_numpy(x))
    codes, scales = ep.Buffer.quantize_int8(t.cuda())
    q, s = front.int8_rows(x)
    assert np.array_equal(host(scales), s) and np.array_equal(host(codes), q)


def _tie_weight(rng, H):
    """fp32 values at and on both sides of ties (q + 1/2) * s, after their
    largest, whose scale s is an odd multiple of 2^-149 in [2^-126, 2^-125)."""
    while True:
        a = F(127) * np.ldexp(F(1 + rng.random()), -126)
        s = a * (F(1) / F(127))
        if 2.0 ** -126 <= s < 2.0 ** -125 and s.view(np.uint32) & 1:
            break
    c = ((rng.integers(0, 126, H) + 0.5) * np.float64(s)).astype(F)
    step = rng.integers(-1, 2, H)
    w = np.where(step < 0, np.nextafter(c, F(0)), np.where(step > 0, np.nextafter(c, F(1)), c))
    w[0] = a
    return w * rng.choice([F(-1), F(1)], H)


@pytest.mark.parametrize("T,H", [(3, 2048), (4099, 264)])
def test_norm_int8_between_the_smallest_scales(T, H):
    """Rows of 1 and -1: the mean square is 1, eps = 2^-60 vanishes and y is the
    weight, in both row shapes."""
    rng = np.random.default_rng(T)
    x = rng.choice([F(-1), F(1)], (T, H))
    xt = torch.from_numpy(x).to(torch.bfloat16).cuda()
    for _ in range(8):
        w = _tie_weight(rng, H)
        _, _, codes, scales = ep.Buffer.add_rmsnorm(xt, None, torch.from_numpy(w).cuda(), 2.0 ** -60, "int8", y=False)
        q, s = front.int8_rows(x * w)
        assert np.array_equal(host(scales), s) and np.array_equal(host(codes), q)
