"""Pins of the plain 64-bit forms of the MoE layer's front: hand-worked cases,
closed forms and central differences (no GPU)."""

from __future__ import annotations

import numpy as np
import pytest

from oracle import front


def test_route_hand_worked_groups():
    # four groups of two; by sums of two, 1.15 and 1.04 beat the group with the best expert (1.0)
    s = np.array([[0.9, 0.1, 0.6, 0.55, 0.2, 0.2, 0.52, 0.52]])
    l = np.log(s / (1 - s))
    idx, w, _ = front.route_scored(l, 3, "sigmoid", bias=np.zeros(8), groups=4, kept=2, top2=True)
    assert idx.tolist() == [[2, 3, 6]]
    idx, w, _ = front.route_scored(l, 3, "sigmoid", bias=np.zeros(8), groups=4, kept=2, top2=False)
    assert idx.tolist() == [[0, 2, 3]]
    assert np.allclose(w, np.array([[0.9, 0.6, 0.55]]) / 2.05)


def test_route_bias_chooses_but_does_not_weigh():
    l = np.array([[0.0, 1.0, 2.0, -1.0]])
    idx, w, s = front.route_scored(l, 2, "softmax", bias=[0, 0, 0, 5.0], renorm=False, scale=2.0)
    assert idx.tolist() == [[3, 2]]
    z = np.exp(l[0])
    assert np.allclose(w[0], 2 * z[[3, 2]] / z.sum()) and np.allclose(s[0], z / z.sum())


def test_route_ties_masks_and_empty_rows():
    inf = np.inf
    l = np.array([[1.0, 1.0, 1.0, 1.0], [-inf, 0.0, np.nan, -inf], [-inf] * 4, [inf, inf, 0, 0]])
    for score in ("softmax", "sigmoid"):
        idx, w, s = front.route_scored(l, 2, score)
        assert idx.tolist() == [[0, 1], [1, -1], [-1, -1], [0, 1]]
        assert np.allclose(w, [[0.5, 0.5], [1, 0], [0, 0], [0.5, 0.5]])
        assert np.all(s[2] == 0) and s[1, 0] == s[1, 2] == 0


def test_route_renormalised_weights_never_underflow():
    l = np.array([[-2000.0, -2001.0, -3000.0]])
    _, w, _ = front.route_scored(l, 2, "sigmoid")
    assert np.allclose(w, [[1 / (1 + np.exp(-1.0)), 1 / (1 + np.exp(1.0))]])


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_gradient_is_the_difference_quotient(score, renorm):
    rng = np.random.default_rng(3)
    T, E, k = 4, 9, 3
    l = rng.normal(size=(T, E))
    l[1, 4] = -np.inf
    gw, gs = rng.normal(size=(T, k)), rng.normal(size=(T, E))
    idx = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
    idx[2, 1] = -1
    idx[3, 2] = idx[3, 0]   # the same expert twice

    def loss(l):
        s = front.route_scores(l, score)
        total = (gs * s).sum()
        for t in range(T):
            ok = [j for j in range(k) if idx[t, j] >= 0 and l[t, idx[t, j]] > -np.inf]
            c = s[t, idx[t, ok]]
            total += 2.5 * (gw[t, ok] * (c / c.sum() if renorm else c)).sum()
        return total

    got, _ = front.route_scored_bwd(l, idx, gw, gs, score, renorm, 2.5)
    for t in range(T):
        for e in range(E):
            if l[t, e] == -np.inf:
                assert got[t, e] == 0
                continue
            d = np.zeros_like(l)
            d[t, e] = 1e-5
            want = (loss(l + d) - loss(l - d)) / 2e-5
            # central differences: error h^2 |f'''| / 6 + 2^-52 |f| / h, both below 1e-8 here
            assert abs(got[t, e] - want) < 1e-7


def test_norm_gradient_is_the_difference_quotient():
    rng = np.random.default_rng(4)
    T, H, eps = 3, 8, 1e-3
    h, w, gy, gh = rng.normal(size=(T, H)), rng.normal(size=H), rng.normal(size=(T, H)), rng.normal(size=(T, H))

    def loss(h, w):
        return (gy * front.rmsnorm(h, w, eps)[0]).sum() + (gh * h).sum()

    gx, gw = front.rmsnorm_bwd(h, w, gy, gh, eps)
    for t in range(T):
        for c in range(H):
            d = np.zeros_like(h)
            d[t, c] = 1e-5
            assert abs(gx[t, c] - (loss(h + d, w) - loss(h - d, w)) / 2e-5) < 1e-7
    for c in range(H):
        d = np.zeros(H)
        d[c] = 1e-5
        assert abs(gw[c] - (loss(h, w + d) - loss(h, w - d)) / 2e-5) < 1e-7


def test_norm_closed_forms():
    y, y32 = front.rmsnorm(np.full((1, 16), 3.0), np.arange(16.0), 0.0)
    assert np.allclose(y, np.arange(16.0)) and y32.dtype == np.float32
    y, _ = front.rmsnorm(np.zeros((1, 8)), np.ones(8), 1e-6)
    assert np.all(y == 0)


def test_int8_rows_hand_worked():
    # amax 127: scale 1, ties to even; zeros: scale 1; not finite: scale NaN, codes 0
    y = np.array([[127, 0.5, 1.5, -2.5, -0.5, 126.4, -127, 3], [0] * 8, [1, np.inf, 0, 0, 0, 0, 0, 0]],
                 np.float32)
    q, s = front.int8_rows(y)
    assert q[0].tolist() == [127, 0, 2, -2, 0, 126, -127, 3]
    assert s[0] == 1 and s[1] == 1 and np.isnan(s[2]) and not q[1:].any()


def test_gemm_int8_exact_and_swiglu():
    x = np.full((1, 131008), -128, np.int8)
    w = np.full((2, 131008), -128, np.int8)
    assert front.gemm_int8(x, [1], w, [1, 0.5]).tolist() == [[128.0 * 128 * 131008, 64.0 * 128 * 131008]]
    assert np.allclose(front.swiglu(np.array([[0.0, 5.0, 20.0, 2.0]])), [[0.0, 40.0 / (1 + np.exp(-20))]])
