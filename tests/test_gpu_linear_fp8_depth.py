"""GPU tests of the FP8 product where its rings in LDS go round: K deep enough that every
buffer of slabs and of scales is used again, for each kernel a size can be given to, with
scales that vary from slab to slab; and operands over the whole range of codes and of
power-of-two scales.

Slabs (128 of K) from which a form's buffers are refilled: 16 or 32 tokens a workgroup
33 and 25 (8 waves, rings of 4 and 3), 64 tokens 13 (4 waves, rings of 3); tiles of
64 x 64 17 (four buffers of four slabs' scales), the other tiles 9 (two buffers).
FORMS holds odd and even numbers of slabs past that, ragged in both directions.

Exact problems (small integers, power-of-two scales) are compared bit for bit.  Others
within: a slab's 128 products, added one at a time in the worst case, each addition
within a step 2 U (whichever way it is rounded) of the magnitudes so far, a slab's own
where its sum is folded into the running one and all slabs' S where the matrix cores add
to that (scales that are powers of two); the fold of each slab; for bf16 results what the
matrix cores cut (test_gpu_linear_fp8); and the result's own rounding."""

from __future__ import annotations

import numpy as np
import pytest
import torch

import combine_ep_plan_amd as ep
from oracle import dense
from tests.gpu_util import host
from tests.test_gpu_linear_fp8 import U, UB, _check, _codes, _cut, _dev, _gpu, _problem  # noqa: F401  (_gpu: fixture)

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32

# (form, M, N, slabs, result); "few": tokens x channels a workgroup
FORMS = [("few 16 x 16", 13, 200, 57, BF), ("few 16 x 16", 16, 331, 50, F32),
         ("few 32 x 16", 21, 4200, 49, BF), ("few 32 x 16", 32, 4203, 50, F32), ("few 32 x 16", 27, 2160, 50, BF),
         ("few 64 x 16", 40, 2100, 25, BF), ("few 64 x 16", 61, 2121, 26, F32),
         ("few 64 x 32", 130, 2100, 15, BF), ("few 64 x 32", 129, 2064, 16, BF), ("few 64 x 32", 131, 2101, 25, F32),
         ("64 x 64", 300, 1701, 33, BF), ("64 x 64", 333, 1712, 34, BF), ("64 x 64", 300, 1700, 35, F32),
         ("128 x 128", 2040, 2017, 17, BF), ("128 x 128", 1900, 2100, 18, BF), ("128 x 128", 2040, 2017, 18, F32),
         ("128 x 128", 1900, 2100, 17, F32),
         ("256 x 256", 3900, 3107, 17, BF), ("256 x 256", 4095, 2952, 18, BF),
         ("128 x 192", 1531, 4091, 17, F32), ("128 x 192", 1536, 4088, 18, F32)]
IDS = [f"{f.replace(' ', '')}-{m}x{n}x{k}-{str(d)[6:]}" for f, m, n, k, d in FORMS]


def _normal(M, N, K, square, pow2, seed=0):
    """Codes and scales of normal values, as the quantiser makes them; results of about 1."""
    rng = np.random.default_rng(M + 7 * N + K + seed)
    x, xs = dense.fp8_blocks(rng.normal(size=(M, K)).astype(np.float32) * np.exp(rng.normal(size=(M, 1))), 1, pow2)
    w, ws = dense.fp8_blocks(rng.normal(size=(N, K)).astype(np.float32), 128 if square else 1, pow2)
    ws = ws * np.exp2(rng.integers(-2, 3, size=ws.shape))   # from slab to slab
    return x, xs, w, (ws * 2.0 ** -round(np.log2(np.sqrt(K)))).astype(np.float32)


def _wide(M, N, K, square):
    """All finite codes; a row's scales 2^-28 .. 2^18 and within 2^2 of each other, so that every slab counts."""
    rng = np.random.default_rng(3 * M + N + K)

    def scales(rows):
        e = rng.integers(-28, 19, size=(rows, 1)) + rng.integers(-2, 3, size=(rows, K // 128))
        return np.exp2(e).astype(np.float32)

    return (_codes(rng, M, K, False), scales(M), _codes(rng, N, K, False), scales(-(-N // 128) if square else N))


def _tolerance(p, square, mag, dtype, pow2):
    slabs = p[0].shape[1] // 128
    return 2 * U * (128 * slabs if pow2 else 128 + 2 * slabs) * mag + (_cut(p, square) if dtype == BF else 0)


def _compare(p, square, dtype, pow2):
    y = host(ep.Buffer.linear_fp8(*_dev(p), out_dtype=dtype, pow2=pow2).double())
    want, mag = dense.linear(*p, square)
    tol = _tolerance(p, square, mag, dtype, pow2)
    err = np.abs(y - want)
    assert np.all(err <= tol + (UB if dtype == BF else U) * (np.abs(want) + tol)), (err / tol).max()


@pytest.mark.parametrize("form,M,N,slabs,dtype", FORMS, ids=IDS)
@pytest.mark.parametrize("square", [True, False])
def test_buffers_used_again_exactly(form, M, N, slabs, dtype, square):
    p = _problem(M, N, slabs * 128, square, True)
    for pow2 in (False, True):
        _check(p, square, dtype, exact=True, pow2=pow2)


@pytest.mark.parametrize("form,M,N,slabs,dtype", FORMS, ids=IDS)
@pytest.mark.parametrize("square", [True, False])
def test_values_of_the_quantisers(form, M, N, slabs, dtype, square):
    for pow2 in (False, True):
        _compare(_normal(M, N, slabs * 128, square, pow2), square, dtype, pow2)


@pytest.mark.parametrize("form,M,N,slabs,dtype", FORMS, ids=IDS)
@pytest.mark.parametrize("square", [True, False])
def test_all_codes_and_wide_scales_of_powers_of_two(form, M, N, slabs, dtype, square):
    p = _wide(M, N, slabs * 128, square)
    for pow2 in (False, True):   # their product lies in fp32's range: the other kernels' too
        _compare(p, square, dtype, pow2)


@pytest.mark.parametrize("form,M,N,slabs", [("few 16 x 16", 13, 208, 57), ("few 32 x 16", 21, 4208, 49),
                                            ("few 64 x 16", 40, 2112, 25), ("few 64 x 32", 130, 2112, 15),
                                            ("64 x 64", 300, 1712, 33), ("128 x 128", 2040, 2016, 17),
                                            ("256 x 256", 3900, 3104, 18)])
@pytest.mark.parametrize("square", [True, False])
def test_swiglu_of_the_quantisers_values(form, M, N, slabs, square):
    """|d silu(g) / dg| <= 1.1; the exponential and the reciprocal within 2^-20."""
    K = slabs * 128
    for pow2 in (False, True):
        p = x, xs, w, ws = _normal(M, N, K, square, pow2)
        y = host(ep.Buffer.linear_fp8(*_dev(p), swiglu=True, pow2=pow2).double())
        out, mag = dense.linear(*p, square)
        tol = _tolerance(p, square, mag, BF, pow2)
        g, u, tg, tu = out[:, 0::2], out[:, 1::2], tol[:, 0::2], tol[:, 1::2]
        s = g / (1 + np.exp(-g))
        want = s * u
        tol = 1.1 * tg * (np.abs(u) + tu) + np.abs(s) * tu + 2.0 ** -20 * np.abs(want)
        err = np.abs(y - want)
        assert np.all(err <= tol + UB * (np.abs(want) + tol) + 1e-37), (err / tol).max()
