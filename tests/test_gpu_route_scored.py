"""GPU parity of scored routing and its backward with the plain 64-bit forms:
ids exact, weights and scores within two fp32 roundings (they are formed in
double and rounded once), gradients within a bound counted from the fp32
operations below."""

from __future__ import annotations

import numpy as np
import pytest
import torch

import combine_ep_plan_amd as ep
from oracle import front
from tests.gpu_util import dev_f32, dev_i32, host, make_group

pytestmark = pytest.mark.gpu
U = 2.0 ** -24      # half a step of fp32
UB = 2.0 ** -8      # of bf16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    ep.load_library()


def _logits(rng, T, E, bf16=False, masked=0.0, std=1.5):
    l = (rng.normal(size=(T, E)) * std).astype(np.float32)
    if masked:
        l[rng.random((T, E)) < masked] = -np.inf
        l[rng.random(T) < masked] = -np.inf
    t = dev_f32(l)
    if bf16:
        t = t.to(torch.bfloat16)
        l = host(t.float())
    return l, t


def _rule(c):
    return ep.RouteRule(score=c["score"], num_groups=c["groups"], kept_groups=c["kept"],
                        group_score="top2" if c["top2"] else "max", renormalise=c["renorm"], scale=c["scale"])


CASES = [dict(T=T, E=E, k=k, groups=g, kept=kept) for T, E, k, g, kept in [
    (1, 256, 8, 8, 4), (3, 8, 2, 1, 1), (129, 65, 3, 5, 2), (64, 60, 6, 10, 3), (50, 5, 7, 1, 1),
    (17, 1024, 16, 64, 33), (33, 1024, 16, 1, 1), (40, 384, 8, 8, 3), (257, 128, 8, 4, 4), (5, 1, 1, 1, 1),
    (70, 64, 1, 64, 7), (31, 100, 16, 4, 1), (1500, 256, 8, 8, 4), (2049, 384, 6, 1, 1), (1025, 130, 4, 2, 1),
    (1030, 64, 8, 16, 5), (1100, 8, 2, 4, 2), (1201, 100, 8, 20, 7), (1301, 192, 16, 48, 9), (1026, 30, 3, 3, 2),
    (1027, 1, 1, 1, 1), (2050, 100, 8, 20, 7), (2050, 96, 16, 48, 9), (4100, 192, 8, 6, 2), (2100, 8, 2, 4, 2),
    (2100, 30, 3, 1, 1)]]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("c", CASES, ids=lambda c: "T{T}E{E}k{k}g{groups}of{kept}".format(**c))
@pytest.mark.parametrize("variant", range(4))
def test_route_scored(c, score, variant):
    c = dict(c, score=score, top2=variant in (1, 2), renorm=variant != 3, scale=(1.0, 2.5, 0.5, 1.0)[variant])
    rng = np.random.default_rng(c["T"] * 7 + c["E"] + variant)
    l, lt = _logits(rng, c["T"], c["E"], bf16=variant == 2, masked=(0, 0, 0.3, 0.1)[variant])
    bias = (rng.normal(size=c["E"]) * 0.2).astype(np.float32) if variant in (1, 3) else None
    h = ep.Handle(make_group(c["E"], 1, 8, c["k"], c["T"], "ht"), c["T"])
    idx, w, s = h.route_scored(lt, _rule(c), None if bias is None else dev_f32(bias), scores=True)
    i2, w2 = h.route_scored(lt, _rule(c), None if bias is None else dev_f32(bias))
    ri, rw, rs = front.route_scored(l, c["k"], score, bias, c["groups"], c["kept"], c["top2"], c["renorm"],
                                    c["scale"])
    assert np.array_equal(host(idx), ri)
    assert np.all(np.abs(host(w) - rw) <= 2 * U * np.abs(rw) + 1e-44)
    assert np.all(np.abs(host(s) - rs) <= 2 * U * rs + 1e-44)
    assert torch.equal(idx, i2) and torch.equal(w, w2)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
def test_ties_masks_and_extremes(score, biased):
    inf, fmax, low = np.inf, np.finfo(np.float32).max, np.finfo(np.float32).min
    E = 8
    l = np.array([[0.5] * E, [0.0, -0.0] * 4, [-inf] * E, [np.nan] * E, [inf] * E, [low] * E, [fmax] * E,
                  [-inf, 1, -inf, 2, np.nan, -inf, -inf, -inf], [low, -inf, low, 3, low, 3, 3, low],
                  [-500, -600, -700, -800, -900, -1000, -1100, -1200], [inf, fmax, 1, -inf, 0, inf, 2, 3],
                  [200, 300, 100, 100, 50, 40, 30, 1e30]], np.float32)
    T = l.shape[0]
    bias = np.zeros(E, np.float32) if biased else None
    for groups, kept, top2, renorm in [(1, 1, False, True), (4, 2, True, True), (2, 1, False, False)]:
        c = dict(score=score, groups=groups, kept=kept, top2=top2, renorm=renorm, scale=1.0)
        h = ep.Handle(make_group(E, 1, 8, 3, T, "ht"), T)
        idx, w, s = h.route_scored(dev_f32(l), _rule(c), None if bias is None else dev_f32(bias), scores=True)
        ri, rw, rs = front.route_scored(l, 3, score, bias, groups, kept, top2, renorm)
        assert np.array_equal(host(idx), ri), (groups, kept, top2)
        assert np.all(np.abs(host(w) - rw) <= 2 * U * np.abs(rw) + 1e-44)
        assert np.all(np.abs(host(s) - rs) <= 2 * U * rs + 1e-44)
        if renorm:   # whatever the logits, the weights of a token with an expert sum to the scale
            some = ri[:, 0] >= 0
            assert np.allclose(host(w)[some].sum(1), 1.0, rtol=4 * U)


def test_bias_masks_and_near_ties():
    """Choices that differ by less than fp32 tells, and biases of -inf and NaN."""
    E, T = 64, 200
    rng = np.random.default_rng(5)
    base = np.float32(0.3)
    l = np.full((T, E), base, np.float32)
    for t in range(T):   # neighbours of one float: sigmoids 1 fp32 step apart or less
        l[t] = base + rng.integers(-3, 4, E).astype(np.float32) * np.spacing(base)
    bias = np.full(E, 0.25, np.float32)
    bias[3], bias[5] = -np.inf, np.nan
    h = ep.Handle(make_group(E, 1, 8, 8, T, "ht"), T)
    for score in ("sigmoid", "softmax"):
        idx, w = h.route_scored(dev_f32(l), ep.RouteRule(score=score), dev_f32(bias))
        # the order of equal biases is the logits' order, ties to the lower expert
        want = np.argsort(-np.where(np.isfinite(bias), l, -np.inf).astype(np.float64), axis=1, kind="stable")[:, :8]
        assert np.array_equal(host(idx), want)


def _bwd_bound(l, mag, bf16, ref):
    """fp32 throughout: an exponential (2 ulp and |x| half steps of its
    argument's rounding), sums of at most 16 + 6 terms in a chain, three
    products and a division: under 96 + 2 |l - lmax| half steps of the
    magnitudes the differences are taken of."""
    lf = np.where(np.isfinite(l), l, 0.0)
    spread = np.abs(lf).max(1, keepdims=True) + np.abs(lf)
    return (96 + 2 * spread) * U * mag + (UB * np.abs(ref) if bf16 else 0.0) + 1e-37


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("with_scores", [True, False])
@pytest.mark.parametrize("T,E,k,bf16", [(1, 256, 8, False), (300, 128, 8, True), (65, 65, 3, False),
                                        (20, 1024, 16, True), (7, 5, 7, False), (4100, 60, 6, False),
                                        (1025, 256, 16, False), (2051, 128, 8, True), (1030, 17, 3, False)])
def test_route_scored_bwd(score, renorm, with_scores, T, E, k, bf16):
    rng = np.random.default_rng(T + E + 2 * renorm + with_scores)
    l, lt = _logits(rng, T, E, bf16=bf16, masked=0.1)
    idx = rng.integers(0, E, (T, k)).astype(np.int32)      # duplicates among them
    idx[rng.random((T, k)) < 0.1] = -1
    gw, gs = rng.normal(size=(T, k)).astype(np.float32), rng.normal(size=(T, E)).astype(np.float32)
    h = ep.Handle(make_group(E, 1, 8, k, T, "ht"), T)
    rule = ep.RouteRule(score=score, renormalise=renorm, scale=2.5)
    got = h.route_scored_bwd(lt, rule, dev_i32(idx), dev_f32(gw), dev_f32(gs) if with_scores else None)
    assert got.dtype == lt.dtype
    ref, mag = front.route_scored_bwd(l, idx, gw, gs if with_scores else None, score, renorm, 2.5)
    g = host(got.float()).astype(np.float64)
    assert np.all(np.abs(g - ref) <= _bwd_bound(l, mag, bf16, ref))
    assert np.all(g[~np.isfinite(l)] == 0)
    assert h.status() == 0


def test_route_bwd_flags_ids_out_of_range():
    l, lt = _logits(np.random.default_rng(1), 4, 16)
    idx = np.array([[0, 1], [16, 2], [-2, 3], [4, 5]], np.int32)
    clean = np.where((idx >= 16) | (idx < 0), -1, idx).astype(np.int32)
    gw = np.ones((4, 2), np.float32) * [[1, 2]]
    h = ep.Handle(make_group(16, 1, 8, 2, 4, "ht"), 4)
    for score in ("softmax", "sigmoid"):
        rule = ep.RouteRule(score=score)
        a = h.route_scored_bwd(lt, rule, dev_i32(clean), dev_f32(gw))
        b = h.route_scored_bwd(lt, rule, dev_i32(idx), dev_f32(gw))
        assert torch.equal(a, b)
    assert h.status() == ep.FLAG_INDEX_RANGE


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_gradient_against_differences_of_the_kernel(score, renorm):
    """The kernel's own weights at l +- d: with d = 2^-6 the central
    difference is off by d^2 f'''/6 (|f'''| of these rational functions of
    scores is below 8 per unit weight) plus two roundings over 2 d."""
    T, E, k, d = 6, 16, 4, 2.0 ** -6
    rng = np.random.default_rng(11)
    l, lt = _logits(rng, T, E)
    rule = ep.RouteRule(score=score, renormalise=renorm)
    g = make_group(E, 1, 8, k, T, "ht")
    h = ep.Handle(g, T)
    idx, w = h.route_scored(lt, rule)
    gw = dev_f32(rng.normal(size=(T, k)))
    grad = host(h.route_scored_bwd(lt, rule, idx, gw))
    order = host(idx)

    def loss(lp):
        # the same experts, whatever order the moved logits put them in
        i, ww = h.route_scored(dev_f32(lp), rule)
        i, ww, o = host(i), host(ww).astype(np.float64), host(gw).astype(np.float64)
        out = np.full(T, np.nan)
        for t in range(T):
            if set(i[t]) == set(order[t]):
                out[t] = sum(o[t, j] * ww[t, list(i[t]).index(order[t, j])] for j in range(k))
        return out

    seen = 0
    for e in range(E):
        p, m = l.copy(), l.copy()
        p[:, e] += np.float32(d)
        m[:, e] -= np.float32(d)
        step = (p[:, e] - m[:, e]).astype(np.float64)
        q = (loss(p) - loss(m)) / step
        ok = np.isfinite(q)
        total = np.abs(host(gw)).sum(1)
        assert np.all(np.abs(q - grad[:, e])[ok] <= total[ok] * (d * d * 8 / 6 + 8 * U / d))
        seen += int(ok.sum())
    assert seen > T * E // 2
