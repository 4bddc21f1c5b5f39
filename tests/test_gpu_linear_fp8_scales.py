"""GPU tests of the FP8 product's power-of-two scales where their product leaves
fp32's range, and of scales that are not powers of two although the caller said so:
the same results from every kernel that a size can be given to.

Codes are small integers (times a power of two), so every sum here is exact in fp32
and the result is the 64-bit form's, rounded once."""

from __future__ import annotations

import numpy as np
import pytest
import torch

import combine_ep_plan_amd as ep
from oracle import dense
from tests.test_gpu_linear_fp8 import _dev, _gpu, _problem  # noqa: F401  (_gpu: fixture)

pytestmark = pytest.mark.gpu

# 16 tokens x 16 channels a workgroup, 32 x 16, 64 x 16, 64 x 32; tiles of 64 x 64, 128 x 128, 256 x 256 (fp32
# results: 128 x 128), fp32 of 128 channels x 192 tokens
FORMS = [(3, 200, 256), (20, 4200, 256), (40, 2100, 256), (130, 2100, 256), (600, 1700, 1152), (2040, 2017, 256),
         (3900, 3100, 256), (1531, 4091, 1152)]


def _run(p, dtype):
    return ep.Buffer.linear_fp8(*_dev(p), pow2=True, out_dtype=dtype).cpu()


@pytest.mark.parametrize("M,N,K", FORMS)
@pytest.mark.parametrize("square", [True, False])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_product_of_the_scales_past_fp32(M, N, K, square, dtype):
    """2^70 * 2^60 over products of 2^-12: results of 2^118 and more, and of nothing where the sum is 0."""
    p = _problem(M, N, K, square, True)
    x, xs, w, ws = p
    small = np.array([0, 0x08, 0x88, 0x10, 0x90], np.uint8)   # 0, +-2^-6, +-2^-5
    rng = np.random.default_rng(M)
    x[:, :128], w[:, :128] = small[rng.integers(0, 5, (M, 128))], small[rng.integers(0, 5, (N, 128))]
    x[::3, :128] = 0
    xs[:, 0], ws[:, 0] = 2.0 ** 70, 2.0 ** 60
    # apart: beside 2^118 the other slabs' integers are below half a step, in 64 bits too
    first, rest = (dense.linear(x[:, c], xs[:, b], w[:, c], ws[:, b], square)[0]
                   for c, b in ((slice(0, 128), slice(0, 1)), (slice(128, None), slice(1, None))))
    want = np.where(first != 0, first, rest)
    assert np.abs(want).max() > 2.0 ** 118
    assert torch.equal(_run(p, dtype), torch.from_numpy(want).to(dtype))


@pytest.mark.parametrize("M,N,K", FORMS)
@pytest.mark.parametrize("square", [True, False])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("of_x", [True, False])
def test_scales_out_of_form_are_taken_at_their_exponent(M, N, K, square, dtype, of_x):
    """3 as 2, -1 as 1, 0 and a subnormal as 2^-127 (nothing beside the other slab's integers), what is
    not finite as NaN."""
    p = _problem(M, N, K, square, True)
    for bad, taken in ((3.0, 2.0), (-1.0, 1.0), (0.75, 0.5), (0.0, 2.0 ** -127), (1e-40, 2.0 ** -127),
                       (np.inf, np.nan), (np.nan, np.nan)):
        given, q = [v.copy() for v in p], [v.copy() for v in p]
        t, at = (1, (M - 1, 1)) if of_x else (3, (min(1, p[3].shape[0] - 1), 1))
        given[t][at], q[t][at] = bad, taken
        want = torch.from_numpy(dense.linear(*q, square)[0])
        y = _run(given, dtype)
        none = want.abs() < 2.0 ** -60
        assert torch.all(y[none].double().abs() <= 2.0 ** -60), bad
        y[none], want[none] = 0, 0
        assert torch.equal(torch.isnan(y), torch.isnan(want)), bad
        assert torch.equal(y.nan_to_num(), want.to(dtype).nan_to_num()), bad


@pytest.mark.parametrize("M,N,K", FORMS)
@pytest.mark.parametrize("square", [True, False])
def test_swiglu_takes_the_same_scales(M, N, K, square):
    """The SwiGLU store's kernels take 3 as 2 too."""
    N = N // 16 * 16
    x, xs, w, ws = _problem(M, N, K, square, True)
    xs[:] = 2.0 ** -4
    xs[M - 1, 1] = 3.0 * 2.0 ** -4
    d = _dev((x, xs, w, ws))
    y = ep.Buffer.linear_fp8(*d, swiglu=True, pow2=True)
    xs[M - 1, 1] = 2.0 ** -3
    assert torch.equal(y, ep.Buffer.linear_fp8(*_dev((x, xs, w, ws)), swiglu=True, pow2=True))
