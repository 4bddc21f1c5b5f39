"""Plain 64-bit forms of the MoE layer's front: scored routing, residual RMS
norm, INT8 rows and the INT8 grouped GEMM (numpy, written from the formulas;
test infrastructure only, it shares no code with the GPU library)."""

from __future__ import annotations

import numpy as np

F32_MAX = float(np.finfo(np.float32).max)


# ---------------------------------------------------------------------------
# scored routing

def clean_logits(logits: np.ndarray) -> np.ndarray:
    """Logits as the routing reads them: NaN masks like -inf, +inf is the largest float."""
    l = np.asarray(logits, np.float64)
    return np.minimum(np.where(np.isnan(l), -np.inf, l), F32_MAX)


def route_scores(l: np.ndarray, score: str) -> np.ndarray:
    live = l > -np.inf
    with np.errstate(over="ignore"):
        if score == "sigmoid":
            return np.where(live, 1.0 / (1.0 + np.exp(-np.where(live, l, 0.0))), 0.0)
        out = np.zeros_like(l)
        for t in range(l.shape[0]):
            m = live[t]
            if m.any():
                z = np.exp(l[t, m] - l[t, m].max())
                out[t, m] = z / z.sum()
        return out


def route_scored(logits, k: int, score="softmax", bias=None, groups=1, kept=1, top2=False,
                 renorm=True, scale=1.0):
    """(idx [T, k], weights float64 [T, k], scores float64 [T, E]), token by token."""
    l = clean_logits(logits)
    T, E = l.shape
    s = route_scores(l, score)
    by_logit = bias is None and not (groups > 1 and top2)
    choice = l.copy() if by_logit else s + (0.0 if bias is None else np.asarray(bias, np.float64))
    choice = np.where((l > -np.inf) & ~np.isnan(choice), choice, -np.inf)
    idx = np.full((T, k), -1, np.int32)
    w = np.zeros((T, k))
    gs = E // groups
    for t in range(T):
        left = choice[t].copy()
        if groups > 1:
            value = np.full(groups, -np.inf)
            for g in range(groups):
                c = sorted((v for v in left[g * gs:(g + 1) * gs] if v > -np.inf), reverse=True)
                if c:
                    value[g] = c[0] + c[1] if top2 and len(c) > 1 else c[0]
            order = sorted(range(groups), key=lambda g: (-value[g], g))
            for g in order[kept:]:
                left[g * gs:(g + 1) * gs] = -np.inf
        for j in range(k):
            e = int(np.argmax(left))   # the first of equals
            if not left[e] > -np.inf:
                break
            idx[t, j] = e
            left[e] = -np.inf
        m = idx[t] >= 0
        if m.any():
            w[t, m] = chosen_shares(l[t, idx[t, m]], score) if renorm else s[t, idx[t, m]]
    return idx, w * scale, s


def chosen_shares(l: np.ndarray, score: str) -> np.ndarray:
    """Chosen scores over their sum, from the scores' logarithms."""
    u = l if score == "softmax" else np.minimum(l, 0.0) - np.log1p(np.exp(-np.abs(l)))
    p = np.exp(u - u.max())
    return p / p.sum()


def route_scored_bwd(logits, idx, gw, gs=None, score="softmax", renorm=True, scale=1.0):
    """Gradient of the logits (float64) and a magnitude per element that its
    rounding errors are relative to."""
    l = clean_logits(logits)
    T, E = l.shape
    s = route_scores(l, score)
    slope = s * (1.0 - s)
    if score == "sigmoid":
        live = l > -np.inf
        with np.errstate(over="ignore"):
            slope = np.where(live, s / (1.0 + np.exp(np.where(live, l, 0.0))), 0.0)
    out, mag = np.zeros((T, E)), np.zeros((T, E))
    for t in range(T):
        ds = np.zeros(E) if gs is None else np.where(l[t] > -np.inf, gs[t], 0.0).astype(np.float64)
        ad = np.abs(ds)   # of the terms: a sum that cancels keeps the rounding errors of its terms
        ok = [j for j in range(idx.shape[1]) if 0 <= idx[t, j] < E and l[t, idx[t, j]] > -np.inf]
        e = idx[t, ok]
        g = np.asarray(gw[t], np.float64)[ok] * scale
        if renorm and len(ok):
            p = chosen_shares(l[t, e], score)
            a = (g * p).sum()
            back = 1.0
            if score == "sigmoid":
                with np.errstate(over="ignore"):
                    back = 1.0 / (1.0 + np.exp(l[t, e]))
            np.add.at(out[t], e, p * (g - a) * back)
            np.add.at(mag[t], e, p * (np.abs(g) + (np.abs(g) * p).sum()) * back)
        else:
            np.add.at(ds, e, g)
            np.add.at(ad, e, np.abs(g))
        if score == "sigmoid":
            out[t] += ds * slope[t]
            mag[t] += ad * slope[t]
        else:
            out[t] += s[t] * (ds - (ds * s[t]).sum())
            mag[t] += s[t] * (ad + (ad * s[t]).sum())
    return out, mag


# ---------------------------------------------------------------------------
# residual RMS norm and 8-bit rows

def rmsnorm(h, w, eps):
    """y in float64 and the fp32 y that the 8-bit codes are decided on:
    (h * w) * rstd with rstd rounded once."""
    h64, w64 = np.asarray(h, np.float64), np.asarray(w, np.float64)
    ms = (h64 * h64).sum(-1, keepdims=True) / h64.shape[-1]
    r = 1.0 / np.sqrt(ms + eps)
    y32 = (np.asarray(h, np.float32) * np.asarray(w, np.float32)) * r.astype(np.float32)
    return h64 * w64 * r, y32


def rmsnorm_bwd(h, w, gy, gh, eps):
    h, w, gy = (np.asarray(a, np.float64) for a in (h, w, gy))
    H = h.shape[-1]
    r = 1.0 / np.sqrt((h * h).sum(-1, keepdims=True) / H + eps)
    n, g = h * r, gy * w
    gx = r * (g - n * (g * n).sum(-1, keepdims=True) / H)
    if gh is not None:
        gx = gx + np.asarray(gh, np.float64)
    return gx, (gy * n).sum(0)


def int8_rows(y32):
    """Codes and fp32 scales of fp32 rows: scale = amax * fp32(1/127), code =
    the integer nearest to the quotient, ties to even."""
    y = np.asarray(y32, np.float32)
    a = np.abs(y).max(-1)
    ok = np.isfinite(y).all(-1)
    s = np.where(a > 0, np.maximum(a * (np.float32(1) / np.float32(127)), np.float32(2.0 ** -126)), np.float32(1))
    s = np.where(ok, s, np.float32(np.nan)).astype(np.float32)
    # the double quotient of two floats is a tie only if the exact one is
    with np.errstate(invalid="ignore"):
        q = np.clip(np.rint(y.astype(np.float64) / s.astype(np.float64)[..., None]), -127, 127)
    return np.where(ok[..., None], q, 0).astype(np.int8), s


# ---------------------------------------------------------------------------
# INT8 grouped product

def gemm_int8(x, sx, w, sw):
    """One group: exact integer sums times both scales, in float64."""
    acc = x.astype(np.int64) @ w.astype(np.int64).T if x.size * w.shape[0] < 1 << 24 else \
        (x.astype(np.float64) @ w.astype(np.float64).T)   # below 2^53: exact too
    return acc.astype(np.float64) * np.asarray(sx, np.float64)[:, None] * np.asarray(sw, np.float64)[None]


def swiglu(h):
    g, u = h[:, 0::2], h[:, 1::2]
    with np.errstate(over="ignore"):
        return g / (1.0 + np.exp(-g)) * u
