"""GPU parity of INT8 rows: the quantiser (codes and scales bit for bit the
64-bit form's), the dispatch of rows that are 8 bits already (a bit copy) and
the grouped INT8 GEMM with its SwiGLU store."""

from __future__ import annotations

import numpy as np
import pytest
import torch

import combine_ep_plan_amd as ep
import oracle
from oracle import front
from tests.gpu_util import dev_f32, dev_i32, host, make_group

pytestmark = pytest.mark.gpu
U, UB = 2.0 ** -24, 2.0 ** -8


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    ep.load_library()
    oracle.build(force=False)


@pytest.mark.parametrize("rows,K", [(1, 8), (1, 64), (5, 520), (300, 2048), (3, 1024), (2, 7168), (3, 8200),
                                    (2, 32768), (4097, 128), (1000, 1536)])
def test_quantize_int8(rows, K):
    rng = np.random.default_rng(rows + K)
    x = rng.normal(size=(rows, K)) * np.exp(rng.normal(size=(rows, 1)) * 4)
    x = torch.from_numpy(x.astype(np.float32)).to(torch.bfloat16).cuda()
    x[rows // 2] = 0
    codes, scales = ep.Buffer.quantize_int8(x)
    q, s = front.int8_rows(host(x.float()))
    assert np.array_equal(host(scales), s) and np.array_equal(host(codes), q)


def test_quantize_int8_ties_and_tiny_rows():
    # amax 127: scale 1, every half-integer a tie; the same rows scaled by powers of two, down to
    # where the scale stops at 2^-126
    v = np.array([127] + [i + 0.5 for i in range(-64, 64)] + [0.25, -0.75] + [0] * 5, np.float32)
    K = v.size
    rows = [v * np.float32(2.0 ** e) for e in (0, 10, -20, 100, -100, -126, -130)]
    x = torch.from_numpy(np.stack(rows)).to(torch.bfloat16)
    codes, scales = ep.Buffer.quantize_int8(x.cuda())
    q, s = front.int8_rows(x.float().numpy())
    assert K % 8 == 0 and np.array_equal(host(scales), s) and np.array_equal(host(codes), q)
    assert np.array_equal(q[0], np.rint(v).astype(np.int8))


def _routing(rng, T, E, k, masked=0.0, hot=None):
    idx = np.stack([rng.permutation(E)[:k] if E >= k else rng.integers(0, E, k) for _ in range(T)]) if T else \
        np.zeros((0, k))
    idx = idx.astype(np.int32).reshape(T, k)
    if hot is not None and T:
        idx[rng.random((T, k)) < 0.6] = hot
    if masked:
        idx[rng.random((T, k)) < masked] = -1
    return idx


def _codes(rng, rows, K):
    c = np.clip(np.rint(rng.normal(size=(rows, K)) * 40), -128, 127).astype(np.int8)
    return c, (rng.random(rows) * 0.03 + 0.001).astype(np.float32)


LAYOUTS = [("ht", 1, 0, 0), ("ll", 1, 5, 0), ("static", 4, 0, 2)]


@pytest.mark.parametrize("layout,R,cap,S", LAYOUTS)
@pytest.mark.parametrize("fmt", ["int8", "fp8"])
@pytest.mark.parametrize("T,H,E,k", [(0, 128, 8, 2), (1, 128, 8, 1), (37, 384, 8, 3), (64, 7168, 16, 8),
                                     (1100, 256, 8, 2), (3000, 1280, 32, 16), (19, 16512, 4, 4)])
def test_dispatch_quantized(layout, R, cap, S, fmt, T, H, E, k):
    if fmt == "int8" and T == 37:
        H = 400   # a multiple of 16 alone
    rng = np.random.default_rng(T + H + k)
    idx = _routing(rng, T, E, k, masked=0.1)
    g = make_group(E, R, H, k, T, layout, cap=cap, S=S)
    h = ep.Handle(g, T)
    h.plan(dev_i32(idx))
    if fmt == "int8":
        c, s = _codes(rng, T, H)
        ct, st = torch.from_numpy(c).cuda(), dev_f32(s)
    else:
        ct = torch.from_numpy(rng.integers(0, 256, (T, H), dtype=np.uint8)).cuda().view(torch.float8_e4m3fn)
        st = dev_f32(rng.random((T, H // 128)))
    w = dev_f32(rng.random((T, k)))
    rows = h.recv_rows
    recv = torch.full((rows, H), 77, dtype=torch.int8, device="cuda").view(ct.dtype)
    rs = torch.full((rows,) + tuple(st.shape[1:]), -5.0, device="cuda")
    ri, rw = torch.empty(rows, dtype=torch.int32, device="cuda"), torch.empty(rows, device="cuda")
    ep.ep_dispatch_quantized(h.ptr, ct, st, w, recv, rs, ri, rw)
    L = oracle.layout(idx, E, layout, cap=cap, R=R, S=S)
    dst = L.dst.reshape(-1)
    used = dst >= 0
    token = np.arange(T * k) // k
    want = np.full((rows, H), 77, np.uint8)
    want[dst[used]] = host(ct.view(torch.uint8))[token[used]]
    ws = np.full(host(rs).shape, -5.0, np.float32)
    ws[dst[used]] = host(st)[token[used]]
    assert np.array_equal(host(recv.view(torch.uint8)), want)   # rows nobody maps to: as they were
    assert np.array_equal(host(rs), ws)
    _, oi, ow = oracle.recv_meta(idx, host(w), L.dst, L.rows)
    assert np.array_equal(host(ri), oi) and np.array_equal(host(rw), ow)


def _groups(h, kind, E, R, cap):
    """(first row, rows, expert, slot index or None) of every group, from the plan's tables."""
    tb = {n: host(v) for n, v in h.tables().items()}
    if kind == "ht":
        return [(int(tb["offsets"][e]), int(tb["counts"][e]), e, None) for e in range(E)]
    if kind == "ll":
        return [(e * cap, min(int(tb["counts"][e]), cap), e, None) for e in range(E)]
    out, C = [], h.rank_rows
    for e in range(E):
        out.append(((e // (E // R)) * C + int(tb["native_row"][e]), int(tb["keep"][e]), e, None))
    for i in range(int(tb["n_segments"][0])):
        e, r, _, n, row = tb["segments"][i]
        s = int(tb["seg_slot"][i])
        out.append((int(r) * C + int(row), int(n), int(e), int(r) * h.group.cfg.slots_per_rank + s if s >= 0 else None))
    return out


def _check_gemm(layout, R, cap, S, T, E, k, K, N, glu, slots=False, hot=None, seed=0):
    rng = np.random.default_rng(T + K + N + seed)
    idx = _routing(rng, T, E, k, masked=0.05, hot=hot)
    g = make_group(E, R, 128, k, T, layout, cap=cap, S=S, mode="inference" if layout == "static" else "training")
    h = ep.Handle(g, T)
    h.plan(dev_i32(idx))
    rows = h.recv_rows
    x, sx = _codes(rng, rows, K)
    w, sw = _codes(rng, E * N, K)
    w, sw = w.reshape(E, N, K), sw.reshape(E, N)
    xt, sxt, wt, swt = torch.from_numpy(x).cuda(), dev_f32(sx), torch.from_numpy(w).cuda(), dev_f32(sw)
    b = ep.Buffer(g)
    slot = slot_s = None
    if slots:   # through the prefetch: poisoned slots, then the plan's copies
        slot = b.prefetch_replicas(wt, h, torch.zeros(R, S, N, K, dtype=torch.int8, device="cuda"))
        slot_s = b.prefetch_replicas(swt, h, torch.full((R, S, N), float("nan"), device="cuda"), scales="row")
    NO = N // 2 if glu else N
    out = torch.full((rows, NO), 9.0, dtype=torch.bfloat16, device="cuda")
    b.expert_gemm_int8(xt, sxt, wt, swt, h, slot, slot_s, out=out, swiglu=glu)
    got = host(out.float()).astype(np.float64)
    covered = np.zeros(rows, bool)
    for row0, n, e, s in _groups(h, layout, E, R, cap):
        if n == 0:
            continue
        covered[row0:row0 + n] = True
        ref = front.gemm_int8(x[row0:row0 + n], sx[row0:row0 + n], w[e], sw[e])
        # exact sums; the conversion, the scales' product and their multiplication round once each
        tol = (UB + 4 * U) * np.abs(ref) + 1e-37
        if glu:
            gate = np.abs(ref[:, 0::2])
            ref = front.swiglu(ref)
            # silu on fp32: the two inputs' errors (the gate's times 1 + |g|), an exponential whose
            # argument and base-2 conversion round (|g| half steps and 2 ulp), a reciprocal, products
            tol = (UB + (24 + 8 * gate) * U) * np.abs(ref) + 1e-37
        assert np.all(np.abs(got[row0:row0 + n] - ref) <= tol), (row0, n, e)
    assert np.all(got[~covered] == 9.0)   # rows no group covers: as they were


@pytest.mark.parametrize("glu", [False, True])
@pytest.mark.parametrize("layout,R,cap,S", [("ht", 1, 0, 0), ("ll", 1, 40, 0), ("static", 4, 0, 2)])
@pytest.mark.parametrize("T,E,k,K,N", [(1, 8, 1, 64, 16), (30, 8, 2, 128, 48), (200, 8, 2, 192, 144),
                                       (300, 4, 3, 320, 272), (64, 16, 8, 1024, 256), (0, 8, 2, 128, 32)])
def test_gemm_int8(layout, R, cap, S, T, E, k, K, N, glu):
    print(f"[gemm int8] {layout} T={T} E={E} k={k} K={K} N={N} glu={glu}", flush=True)
    _check_gemm(layout, R, cap, S, T, E, k, K, N, glu, hot=2 if T == 300 else None)


# many rows an expert and N >= 256: the large tiles; full, short and single-row tails
@pytest.mark.parametrize("glu", [False, True])
@pytest.mark.parametrize("T,E,k,K,N,hot", [(1030, 4, 2, 64, 256, None), (1500, 4, 2, 128, 272, 1),
                                           (700, 4, 4, 192, 512, 3), (520, 2, 2, 1088, 336, None),
                                           (4096, 8, 1, 640, 256, 5)])
def test_gemm_int8_large_groups(T, E, k, K, N, hot, glu):
    print(f"[gemm int8] T={T} E={E} k={k} K={K} N={N} glu={glu}", flush=True)
    _check_gemm("ht", 1, 0, 0, T, E, k, K, N, glu, hot=hot)


# tiles of 65 to 128 rows, and shorter ones beside them; one to nine slabs of K
@pytest.mark.parametrize("glu", [False, True])
@pytest.mark.parametrize("layout,cap,T,E,k,K,N,hot", [
    ("ht", 0, 190, 4, 2, 64, 256, None), ("ht", 0, 190, 4, 2, 128, 272, 1), ("ht", 0, 220, 4, 2, 192, 512, None),
    ("ll", 128, 200, 4, 2, 256, 288, None), ("ht", 0, 230, 4, 2, 1088, 336, 3), ("ht", 0, 70, 1, 1, 384, 256, None),
    ("ll", 66, 400, 2, 1, 448, 256, None), ("ht", 0, 160, 64, 8, 256, 1024, 5)])
def test_gemm_int8_half_tiles(layout, cap, T, E, k, K, N, hot, glu):
    print(f"[gemm int8] {layout} T={T} E={E} k={k} K={K} N={N} glu={glu}", flush=True)
    _check_gemm(layout, 1, cap, 0, T, E, k, K, N, glu, hot=hot)


@pytest.mark.parametrize("N", [1, 7, 20, 100, 257, 300])
def test_gemm_int8_odd_columns(N):
    _check_gemm("ht", 1, 0, 0, 150, 4, 2, 192, N, False)
    _check_gemm("ht", 1, 0, 0, 600, 2, 2, 192, N, False)


@pytest.mark.parametrize("glu", [False, True])
def test_gemm_int8_through_slots(glu):
    _check_gemm("static", 4, 0, 2, 400, 8, 2, 256, 64, glu, slots=True, hot=0)
    _check_gemm("static", 4, 0, 1, 1200, 8, 2, 256, 256, glu, slots=True, hot=7)


@pytest.mark.parametrize("T", [3, 600])
def test_gemm_int8_sums_are_exact(T):
    """The largest K and codes: sums near 2^31, exact in 32 bits (fp32 would
    lose 7 of them); K = 131008, the largest multiple of 64 served."""
    K, N, E = 131008, 256 if T == 600 else 16, 2
    h = ep.Handle(make_group(E, 1, 128, 1, T, "ht"), T)
    h.plan(dev_i32(np.arange(T).reshape(T, 1) % E))
    x = torch.full((T, K), -128, dtype=torch.int8, device="cuda")
    x[:, 1] = 127
    w = torch.full((E, N, K), -128, dtype=torch.int8, device="cuda")
    w[1] = 127
    one = torch.ones(T, device="cuda")
    # scales that take the sum's leading part away are not possible in one product, so the sum is
    # read through bf16: exact sums and sums off by one step of bf16 differ
    out = ep.Buffer(h.group).expert_gemm_int8(x, one, w, torch.ones(E, N, device="cuda"), h)
    lead = [128 * 128 * (K - 1) - 127 * 128, -128 * 127 * (K - 1) + 127 * 127]
    off = host(h.tables()["offsets"])
    for e in range(E):
        v = torch.tensor(float(np.float32(lead[e]))).to(torch.bfloat16).item()
        assert torch.all(out[off[e]:off[e + 1]].float() == v)


def test_gemm_int8_small_sums_bit_for_bit():
    """Sums below 2^8 with unit scales are bf16 values: equality."""
    rng = np.random.default_rng(6)
    for T, N in ((100, 64), (900, 256)):
        E, K = 4, 256
        idx = _routing(rng, T, E, 2)
        h = ep.Handle(make_group(E, 1, 128, 2, T, "ht"), T)
        h.plan(dev_i32(idx))
        x = (rng.random((h.recv_rows, K)) < 0.2).astype(np.int8) * rng.integers(-1, 2, (h.recv_rows, K)).astype(np.int8)
        w = rng.integers(-2, 3, (E, N, K)).astype(np.int8)
        out = ep.Buffer(h.group).expert_gemm_int8(torch.from_numpy(x).cuda(), torch.ones(h.recv_rows, device="cuda"),
                                                  torch.from_numpy(w).cuda(), torch.ones(E, N, device="cuda"), h)
        off = host(h.tables()["offsets"])
        for e in range(E):
            ref = x[off[e]:off[e + 1]].astype(np.int64) @ w[e].astype(np.int64).T
            assert np.abs(ref).max() <= 256
            assert np.array_equal(host(out[off[e]:off[e + 1]].float()), ref)


def test_gemm_int8_silu_extremes():
    """Gates far below and above: the activation's whole range, one rounding."""
    E, T, K, N = 1, 64, 64, 32
    h = ep.Handle(make_group(E, 1, 128, 1, T, "ht"), T)
    h.plan(dev_i32(np.zeros((T, 1))))
    x = np.zeros((T, K), np.int8)
    x[:, 0], x[:, 1] = 1, 1
    w = np.zeros((E, N, K), np.int8)
    w[0, 0::2, 0] = np.arange(16) * 8 - 127          # gates -127 .. -7, then scaled by the row
    w[0, 1::2, 1] = 100
    sx = np.linspace(0.01, 1.5, T).astype(np.float32)
    out = ep.Buffer(h.group).expert_gemm_int8(torch.from_numpy(x).cuda(), dev_f32(sx), torch.from_numpy(w).cuda(),
                                              torch.ones(E, N, device="cuda"), h, swiglu=True)
    ref64 = front.gemm_int8(x, sx, w[0], np.ones(N))
    ref = front.swiglu(ref64)
    tol = (UB + (24 + 8 * np.abs(ref64[:, 0::2])) * U) * np.abs(ref) + 2.0 ** -133   # bf16's smallest step
    assert np.all(np.abs(host(out.float()).astype(np.float64) - ref) <= tol)


def test_calls_refuse_tensors_they_cannot_take():
    x = torch.zeros(8, 64, dtype=torch.bfloat16, device="cuda")
    q, s = torch.empty(8, 64, dtype=torch.int8, device="cuda"), torch.empty(8, device="cuda")
    with pytest.raises(ValueError, match="contiguous"):
        ep.ep_quantize_int8(x[:, ::2], q[:, :32].contiguous(), s)
    with pytest.raises(ValueError, match="on the GPU"):
        ep.ep_quantize_int8(x, q, s.cpu())
    with pytest.raises(TypeError, match="dtype"):
        ep.ep_quantize_int8(x.half(), q, s)
    with pytest.raises(ep.EpError, match="BAD_SHAPE"):
        ep.ep_quantize_int8(x, q, s[:7])
    with pytest.raises(ep.EpError, match="INVALID_ARG"):   # rows start at 16-byte boundaries
        ep.ep_quantize_int8(x.view(-1)[4:4 + 7 * 64].view(7, 64), q[:7], s[:7])
    # a stream by object and by address; recorded
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for st in (side, side.cuda_stream):
        s.fill_(-1)
        side.wait_stream(torch.cuda.current_stream())
        ep.ep_quantize_int8(x, q, s, stream=st)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.all(s == 1)
