"""GPU parity of the block quantiser: codes and scales bit for bit, rows and
columns, both block forms and scale formats."""

from __future__ import annotations

import numpy as np
import pytest
import torch

import combine_ep_plan_amd as ep
from oracle import dense
from tests.gpu_util import host

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    ep.load_library()


def _matrix(R, C, seed=0):
    rng = np.random.default_rng(R * 7 + C + seed)
    v = rng.normal(size=(R, C)) * np.exp(rng.normal(size=(R, 1)) * 2) * np.exp(rng.normal(size=C))
    if R > 3:
        v[2] = 0                       # a row of zeros
    v[:, 5] = 0                        # a column of zeros
    v[0, 6], v[R - 1, C - 1] = -0.0, 1e-38
    return torch.from_numpy(v.astype(np.float32)).to(torch.bfloat16)


def _check(x, got, block, pow2):
    codes, scales, codes_t, scales_t = got
    v = x.float().numpy()
    R, C = v.shape
    rows = 128 if block == "square" else 1
    Rp = -(-R // 128) * 128
    if codes is not None:
        c, s = dense.fp8_blocks(v, rows, pow2)
        assert np.array_equal(host(codes.view(torch.uint8)), c)
        assert np.array_equal(host(scales), s, equal_nan=True)
    if codes_t is not None:
        t = np.zeros((C, Rp), np.float32)
        t[:, :R] = v.T
        c, s = dense.fp8_blocks(t, rows, pow2)
        c[:, R:] = 0
        assert np.array_equal(host(codes_t.view(torch.uint8)), c)
        assert np.array_equal(host(scales_t), s, equal_nan=True)


@pytest.mark.parametrize("R,C", [(1, 128), (7, 256), (127, 128), (128, 384), (129, 128), (300, 640), (2049, 1152)])
@pytest.mark.parametrize("block", ["rows", "square"])
@pytest.mark.parametrize("pow2", [False, True])
def test_quantize_2d(R, C, block, pow2):
    x = _matrix(R, C)
    xd = x.cuda()
    _check(x, ep.Buffer.quantize_fp8_2d(xd, block, pow2=pow2), block, pow2)
    _check(x, ep.Buffer.quantize_fp8_2d(xd, block, transposed=False, pow2=pow2), block, pow2)
    _check(x, ep.Buffer.quantize_fp8_2d(xd, block, rows=False, pow2=pow2), block, pow2)


def test_rows_are_the_row_quantisers():
    x = _matrix(257, 1024).cuda()
    for pow2 in (False, True):
        c, s, _, _ = ep.Buffer.quantize_fp8_2d(x, "rows", transposed=False, pow2=pow2)
        c2, s2 = ep.Buffer.quantize_fp8(x, pow2=pow2)
        assert torch.equal(c.view(torch.uint8), c2.view(torch.uint8)) and torch.equal(s, s2)


def test_a_squares_transpose_is_the_same_codes():
    x = _matrix(256, 512).cuda()
    c, s, ct, st = ep.Buffer.quantize_fp8_2d(x, "square")
    assert torch.equal(c.view(torch.uint8).t(), ct.view(torch.uint8)) and torch.equal(s.t(), st)


@pytest.mark.parametrize("block", ["rows", "square"])
def test_blocks_that_are_not_finite_tiny_or_huge(block):
    x = _matrix(260, 384)
    x[3, 7], x[140, 130], x[259, 383] = float("inf"), float("nan"), float("-inf")
    x[10, 256:] = 1e-39      # subnormal bf16 values: scales below 2^-80 divide
    x[11, 256:] = 3e38
    _check(x, ep.Buffer.quantize_fp8_2d(x.cuda(), block), block, False)
    y = torch.full((128, 128), 9.2e-41, dtype=torch.bfloat16)
    y[::3] = -9.2e-41
    for pow2 in (False, True):
        _check(y, ep.Buffer.quantize_fp8_2d(y.cuda(), block, pow2=pow2), block, pow2)


def test_empty_other_stream_and_captured():
    got = ep.Buffer.quantize_fp8_2d(torch.empty(0, 256, device="cuda", dtype=torch.bfloat16))
    assert got[0].shape == (0, 256) and got[2].shape == (256, 0)
    x = _matrix(300, 512).cuda()
    want = ep.Buffer.quantize_fp8_2d(x)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    other = ep.Buffer.quantize_fp8_2d(x, stream=s)
    s.synchronize()
    assert all(torch.equal(p.view(torch.uint8), q.view(torch.uint8)) for p, q in zip(want, other))
    out = [torch.zeros_like(t) for t in want]
    step = ep.prepare(lambda: ep.ep_quantize_fp8_2d(x, *out))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ep.ep_quantize_fp8_2d(x, *out)
    for i in range(3):
        x.copy_(_matrix(300, 512, i + 1))
        want = ep.Buffer.quantize_fp8_2d(x)
        for run in (graph.replay, step):
            for t in out:
                t.view(torch.uint8).zero_()
            run()
            assert all(torch.equal(p.view(torch.uint8), q.view(torch.uint8)) for p, q in zip(want, out))


def test_two_dimensional_only():
    with pytest.raises(ep.EpError):
        x = torch.zeros(2, 2, 128, device="cuda", dtype=torch.bfloat16)
        ep.ep_quantize_fp8_2d(x, x.to(torch.float8_e4m3fn), torch.zeros(4, 1, device="cuda"), None, None)


@pytest.mark.parametrize("block", ["rows", "square"])
def test_offsets_past_32_bits(block):
    """A matrix of more than 2^32 values: its last tile as it is alone."""
    R, C = 65700, 65536
    x = torch.zeros(R, C, dtype=torch.bfloat16, device="cuda")
    last = torch.randn(R % 128, 128, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    x[-last.shape[0]:, -128:] = last
    got = ep.Buffer.quantize_fp8_2d(x, block)
    want = ep.Buffer.quantize_fp8_2d(last, block)
    u8 = lambda t: t.view(torch.uint8)  # noqa: E731
    n = last.shape[0] if block == "rows" else 1
    assert torch.equal(u8(got[0])[-last.shape[0]:, -128:], u8(want[0])) and torch.equal(got[1][-n:, -1:], want[1])
    assert torch.equal(u8(got[2])[-128:, -128:], u8(want[2])) and torch.equal(got[3][-want[3].shape[0]:, -1:], want[3])
    assert not u8(got[0])[:, 0].any() and not u8(got[2])[0].any()
