"""The 64-bit forms of the layer's dense half, held against published vectors,
torch's own CPU routines, differences and closed forms."""

from __future__ import annotations

import numpy as np
import pytest
import torch

from oracle import dense


def test_philox_known_answers():
    """The known-answer vectors published with the generator."""
    z = dense.philox((0, 0, 0, 0), (0, 0))
    assert z == (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)
    f = 0xFFFFFFFF
    assert dense.philox((f, f, f, f), (f, f)) == (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)
    assert dense.philox((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0)) == (
        0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1)


def test_dropout_bits_are_the_generators_halves():
    seed, offset = 0x0123456789ABCDEF, 0xFEDCBA9876543210
    bits = dense.dropout_bits(43, seed, offset)
    for i in range(43):
        c = dense.philox((i // 8, 0, offset & dense.M32, offset >> 32), (seed & dense.M32, seed >> 32))
        w = c[i % 8 // 2]
        assert bits[i] == (w >> 16 if i % 2 else w & 0xFFFF)


def test_dropout_factor_is_unbiased():
    """The mean of 2^20 factors is 1 within six standard deviations."""
    n = 1 << 20
    for p in (0.1, 0.5, 0.9):
        f = dense.dropout_factor((n,), p, 7, 1)
        assert abs(f.mean() - 1) < 6 * np.sqrt(p / (1 - p) / n)
    assert np.all(dense.dropout_factor((64,), 0.0, 1, 2) == 1) and np.all(dense.dropout_factor((64,), 1.0, 1, 2) == 0)


@pytest.mark.parametrize("bias", [False, True])
def test_layernorm_against_torch(bias):
    rng = np.random.default_rng(1)
    h, w, b = rng.normal(size=(5, 24)) + 3, rng.normal(size=24), rng.normal(size=24)
    gy, gh = rng.normal(size=(5, 24)), rng.normal(size=(5, 24))
    th, tw, tb = (torch.from_numpy(v).requires_grad_() for v in (h, w, b))
    y = torch.nn.functional.layer_norm(th, (24,), tw, tb if bias else None, 1e-3)
    (y * torch.from_numpy(gy)).sum().backward()
    assert np.allclose(dense.layernorm(h, w, b if bias else None, 1e-3)[0], y.detach().numpy(), rtol=1e-12, atol=1e-12)
    g, gw, gb = dense.layernorm_bwd(h, w, gy, gh, 1e-3)
    assert np.allclose(g - gh, th.grad.numpy(), rtol=1e-10, atol=1e-12)
    assert np.allclose(gw, tw.grad.numpy(), rtol=1e-12)
    assert np.allclose(gb, gy.sum(0))


def test_layernorm_gradients_against_differences():
    rng = np.random.default_rng(2)
    h, w, gy = rng.normal(size=(2, 8)), rng.normal(size=8), rng.normal(size=(2, 8))
    f = lambda a, c: (dense.layernorm(a, c, None, 1e-2)[0] * gy).sum()  # noqa: E731
    g, gw, _ = dense.layernorm_bwd(h, w, gy, None, 1e-2)
    d = 1e-6
    for i in range(2):
        for j in range(8):
            e = np.zeros_like(h)
            e[i, j] = d
            assert abs((f(h + e, w) - f(h - e, w)) / (2 * d) - g[i, j]) < 1e-7
    for j in range(8):
        e = np.zeros(8)
        e[j] = d
        assert abs((f(h, w + e) - f(h, w - e)) / (2 * d) - gw[j]) < 1e-7


def test_layernorm_closed_forms():
    y, n, r = dense.layernorm(np.array([[1.0, 3.0, 1.0, 3.0], [5.0, 5.0, 5.0, 5.0]]), np.ones(4), np.full(4, 2.0), 0.0 + 1e-30)
    assert np.allclose(y[0], [1, 3, 1, 3]) and np.allclose(y[1], 2.0)


@pytest.mark.parametrize("rows", [1, 128])
@pytest.mark.parametrize("pow2", [False, True])
def test_fp8_blocks(rows, pow2):
    rng = np.random.default_rng(3)
    v = rng.normal(size=(130, 256)).astype(np.float32)
    v[3] = 0
    v[129, :128] = 0 if rows == 1 else v[129, :128]
    c, s = dense.fp8_blocks(v, rows, pow2)
    assert s.shape == (130 if rows == 1 else 2, 2)
    back = dense.fp8_values(c, s, rows)
    step = np.repeat(np.repeat(s, rows, 0)[:130], 128, 1).astype(np.float64)
    assert np.all(np.abs(back - v) <= 2.0 ** -4 * np.abs(v) * (1 + 2.0 ** -20) + step * 2.0 ** -10)
    if pow2:
        assert np.all(np.frexp(s)[0] == 0.5)
    elif rows == 1:
        assert s[3, 0] == 1.0 and np.all(c[3] == 0)
    v[5, 5] = np.inf
    c, s = dense.fp8_blocks(v, rows, pow2)
    assert np.isnan(s[5 if rows == 1 else 0, 0]) and np.all(c[5, :128] == 0) and np.isfinite(s[:, 1]).all()


def test_linear_against_decoded_matmul():
    rng = np.random.default_rng(4)
    x, xs = dense.fp8_blocks(rng.normal(size=(3, 256)), 1, False)
    for rows in (1, 128):
        w, ws = dense.fp8_blocks(rng.normal(size=(130, 256)), rows, False)
        want = np.zeros((3, 130))
        tx = torch.from_numpy(x).view(torch.float8_e4m3fn).double().numpy()
        tw = torch.from_numpy(w).view(torch.float8_e4m3fn).double().numpy()
        for m in range(3):
            for n in range(130):
                for b in range(2):
                    t = tx[m, 128 * b:128 * b + 128] @ tw[n, 128 * b:128 * b + 128]
                    want[m, n] += t * float(xs[m, b]) * float(ws[n // rows, b])
        assert np.allclose(dense.linear(x, xs, w, ws, rows == 128)[0], want, rtol=1e-12, atol=1e-12)
