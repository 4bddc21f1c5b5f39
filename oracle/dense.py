"""Plain 64-bit forms of a layer's dense half: dropout from a counter-based
generator, residual layer norm and its gradients, FP8 blocks, and the FP8 product
with a scale per block of 128 (numpy, written from the formulas; test
infrastructure only, it shares no code with the GPU library)."""

from __future__ import annotations

import numpy as np
import torch

M32 = 0xFFFFFFFF


def philox(counter: tuple, key: tuple) -> tuple:
    """Philox4x32-10 of one counter (four words) and key (two words), in
    Python's integers (Salmon et al., 2011, section 4.3)."""
    c, k = list(counter), list(key)
    for _ in range(10):
        p, q = 0xD2511F53 * c[0], 0xCD9E8D57 * c[2]
        c = [(q >> 32) ^ c[1] ^ k[0], q & M32, (p >> 32) ^ c[3] ^ k[1], p & M32]
        k = [(k[0] + 0x9E3779B9) & M32, (k[1] + 0xBB67AE85) & M32]
    return tuple(c)


def dropout_bits(n: int, seed: int, offset: int) -> np.ndarray:
    """The 16 bits of values 0 .. n - 1 (uint16): all counters at once."""
    b = np.arange((n + 7) // 8, dtype=np.uint64)
    word = lambda v, s: np.uint64((v >> s) & M32)  # noqa: E731
    lo = np.uint64(M32)
    x = [b & lo, b >> np.uint64(32), np.full_like(b, word(offset, 0)), np.full_like(b, word(offset, 32))]
    k0, k1 = int(word(seed, 0)), int(word(seed, 32))
    for _ in range(10):
        p, q = x[0] * np.uint64(0xD2511F53), x[2] * np.uint64(0xCD9E8D57)
        x = [(q >> np.uint64(32)) ^ x[1] ^ np.uint64(k0), q & lo, (p >> np.uint64(32)) ^ x[3] ^ np.uint64(k1), p & lo]
        k0, k1 = (k0 + 0x9E3779B9) & M32, (k1 + 0xBB67AE85) & M32
    halves = [h for w in x for h in (w & np.uint64(0xFFFF), w >> np.uint64(16))]
    return np.stack(halves, 1).astype(np.uint16).reshape(-1)[:n]


def dropout_factor(shape: tuple, p: float, seed: int, offset: int) -> np.ndarray:
    """0 for what is dropped, fp32(65536 / threshold) for what stays (float64)."""
    stay = int(np.floor((1 - p) * 65536 + 0.5))
    bits = dropout_bits(int(np.prod(shape)), seed, offset)
    return np.where(bits < stay, float(np.float32(65536 / max(stay, 1))), 0.0).reshape(shape)


def layernorm(h: np.ndarray, w: np.ndarray, b: np.ndarray | None, eps: float):
    """(y, n, rstd) of rows, in float64."""
    h = np.asarray(h, np.float64)
    d = h - h.mean(1, keepdims=True)
    r = 1.0 / np.sqrt((d * d).mean(1, keepdims=True) + eps)
    y = d * r * np.asarray(w, np.float64)
    return (y if b is None else y + np.asarray(b, np.float64)), d * r, r


def layernorm_bwd(h, w, gy, gh, eps):
    """(grad, grad_weight, grad_bias) in float64; grad joined with gh if given."""
    _, n, r = layernorm(h, w, None, eps)
    gy = np.asarray(gy, np.float64)
    g = gy * np.asarray(w, np.float64)
    grad = r * (g - g.mean(1, keepdims=True) - n * (g * n).mean(1, keepdims=True))
    return (grad if gh is None else grad + np.asarray(gh, np.float64)), (gy * n).sum(0), gy.sum(0)


def fp8_blocks(v: np.ndarray, rows: int, pow2: bool):
    """e4m3 codes (uint8) and fp32 scales of a float32 matrix by blocks of
    ``rows`` x 128; a block that is not finite has codes 0 and a NaN scale."""
    v = np.asarray(v, np.float32)
    R, C = v.shape
    Rb = -(-R // rows)
    codes, scales = np.zeros((R, C), np.uint8), np.ones((Rb, C // 128), np.float32)
    full = np.zeros((Rb * rows, C), np.float32)
    full[:R] = v
    blocks = full.reshape(Rb, rows, C // 128, 128).transpose(0, 2, 1, 3)
    a = np.abs(blocks).max((2, 3))
    with np.errstate(invalid="ignore", over="ignore"):
        s = np.where(a > 0, np.maximum(a / np.float32(448), np.float32(2.0 ** -149)), np.float32(1)).astype(np.float32)
        if pow2:
            e = np.ceil(np.log2(s.astype(np.float64), where=np.isfinite(s), out=np.zeros(s.shape)))
            s = np.where(a > 0, np.maximum(np.exp2(e), 2.0 ** -126), 1).astype(np.float32)
    bad = ~np.isfinite(a)
    s[bad] = np.nan
    with np.errstate(invalid="ignore", over="ignore"):
        q = np.clip(blocks / s[:, :, None, None], -448, 448).astype(np.float32)
    q[bad] = 0.0
    enc = torch.from_numpy(np.ascontiguousarray(q)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    codes = enc.transpose(0, 2, 1, 3).reshape(Rb * rows, C)[:R]
    scales = s
    return np.ascontiguousarray(codes), scales


def fp8_values(codes: np.ndarray, scales: np.ndarray, rows: int) -> np.ndarray:
    """What codes (uint8) and scales stand for, in float64."""
    v = torch.from_numpy(np.ascontiguousarray(codes)).view(torch.float8_e4m3fn).double().numpy()
    s = np.repeat(np.repeat(np.asarray(scales, np.float64), rows, 0)[:v.shape[0]], 128, 1)
    return v * s


def linear(x, xs, w, ws, square: bool, addend=None, swiglu: bool = False):
    """(out, sum of the terms' magnitudes) in float64."""
    a, b = fp8_values(x, xs, 1), fp8_values(w, ws, 128 if square else 1)
    out, mag = a @ b.T, np.abs(a) @ np.abs(b).T
    if swiglu:
        g, u = out[:, 0::2], out[:, 1::2]
        return g / (1.0 + np.exp(-g)) * u, mag
    return (out if addend is None else out + np.asarray(addend, np.float64)), mag
