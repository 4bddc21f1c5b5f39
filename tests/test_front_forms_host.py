"""The cases of ``test_gpu_front_forms.py`` reach every compiled form of the
front's kernels, by the launch rules as the sources have them."""

from __future__ import annotations

import re

import combine_ep_plan_amd as ep
from tests import front_forms as ff


def _compiled(kernel: str) -> set:
    """Template arguments of a kernel in the built library: numbers, and t / f for uint16 / float."""
    with open(ep.library_path(), "rb") as fh:
        blob = fh.read()
    name = f"_ZN3epk{len(kernel)}{kernel}".encode()
    out = set()
    for args in set(re.findall(name + rb"I((?:[tf]|L[bil]\d+E)+)E", blob)):
        out.add(tuple(int(a[2:-1]) if a[:1] == b"L" else a.decode() for a in re.findall(rb"[tf]|L[bil]\d+E", args)))
    assert out, kernel
    return out


def test_streaming_gemm():
    got = set()
    for layout, R, cap, S, T, E, k, K, N, hot, want in ff.STREAM_CASES:
        for glu in (False, True):
            form = ff.gemm_int8_form(layout, T, E, k, cap, K, N, glu)
            assert form == ("stream", glu) + want, (layout, T, E, k, K, N, form)
            got.add(tuple(int(v) for v in form[1:]))
    assert got == _compiled("k_grouped_gemm_i8_stream")
    # six entries in ten are the hot expert's: more rows than one pass over the weights takes
    hot = {(c[10], c[0]) for c in ff.STREAM_CASES if c[9] is not None and 0.5 * c[4] * c[6] > ff.SHORT_ROWS}
    assert {("ht", f) for f in {c[10] for c in ff.STREAM_CASES}} <= {(l, f) for f, l in hot}


def test_large_and_small_tiles():
    n, E = sum(ff.WIDE_ROWS), len(ff.WIDE_ROWS)
    for K, N in ff.WIDE_CASES:
        assert ff.gemm_int8_form("ht", n, E, 1, 0, K, N, True) == ("wide", True)
    for K, N in ff.TILE_CASES:
        assert ff.gemm_int8_form("ht", n, E, 1, 0, K, N, True) == ("tiles", True)
    assert _compiled("k_grouped_gemm_i8_256") == _compiled("k_grouped_gemm_i8") == {(0,), (1,)}
    slabs = {-(-K // 128) for K, _ in ff.WIDE_CASES}
    assert {1, 2, 3, 4} <= slabs and {K % 128 for K, _ in ff.WIDE_CASES} == {0, 64}


def test_norm_and_quantiser():
    forms = {ff.row_form(T, H) for T, H in ff.ROW_CASES}
    assert {(v, int(w)) for v, w, _ in forms} == _compiled("k_quantize_int8")
    assert {a for a in _compiled("k_add_rmsnorm")} == {
        (t, r, v, int(w)) for v, w, _ in forms for t, r in (("t", 0), ("t", 1), ("f", 1))}
    assert {(2, 256), (2, 512), (2, 1024), (4, 1024)} <= {(v, th) for v, w, th in forms if not w}
    assert any(T % 4 for T, H in ff.ROW_CASES if ff.row_form(T, H)[1])   # a workgroup not full of rows


def test_scored_routing():
    got = {(t,) + ff.route_form(T, E, ff.MANY_FORWARD) for T, E, *_ in ff.ROUTE_CASES for t in "tf"}
    assert got == _compiled("k_score_route")
    got = {(t, d) + ff.route_form(T, E, ff.MANY_BACKWARD)
           for T, E, _ in ff.ROUTE_BWD_CASES for t in "tf" for d in (0, 1)}
    assert got == _compiled("k_score_route_bwd")
    for rows in (ff.ROUTE_CASES, ff.ROUTE_BWD_CASES):   # waves and workgroups not full of tokens
        assert any(T % 16 for T, E, *_ in rows if ff.route_form(T, E, 128)[0] == 16)


def test_dispatch_stores():
    got = {ff.stores_form(k, T * k, H + 4, s) for T, H, k, s in ff.STORE_CASES}
    assert {(k, int(nt)) for k, nt in got} == _compiled("k_dispatch_rows8")
    auto = {ff.stores_form(k, T * k, H + 4, s)[1] for T, H, k, s in ff.STORE_CASES if s == "auto"}
    assert auto == {False, True}
