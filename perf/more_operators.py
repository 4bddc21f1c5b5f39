"""Measured operators of a layer's dense half: residual layer norm with dropout
and 8-bit rows and its backward, dropout from a counter-based generator, FP8
products with a scale per block of 128, and the quantiser that feeds them.

``run`` computes them as elementary torch operations, or with ``own`` by the
library's entry points.  Both take the inputs ``prepare`` makes; a state holds
its inputs, its output buffers and (``own``) the workspace a program keeps."""

import math

import numpy as np
import torch

own = False

# The shapes are this repository's workloads: decode (T 128, H 7168), prefill
# (T 4096, H 7168), training (T 16384, H 4096, experts of 1536 channels).
EPS = 1e-5


def _ln(T, H, **kw):
    c = dict(op="ln", T=T, H=H, residual="bf16", wfp32=False, bias=True, p=0.0, y=True, quant="none")
    c.update(kw)
    return c


def _linear(M, N, K, **kw):
    c = dict(op="linear", M=M, N=N, K=K, wscale="block", out="bf16", add=False, swiglu=False, pow2=False)
    c.update(kw)
    return c


def listed():
    return [
        # a decode step's norm: residual added, bf16 rows for the router and FP8 rows for the products
        dict(_ln(128, 7168, quant="fp8"), name="ln_decode_fp8"),
        # a training step's: the branch is dropped out, joins the stream and is normalised
        dict(_ln(16384, 4096, p=0.1), name="ln_training_dropout"),
        # its backward, the stream's own gradient joining; gradients of branch, stream, weight and bias
        dict(_ln(16384, 4096, op="ln_bwd", p=0.1), name="ln_bwd_training_dropout"),
        # a small fine-tuning batch of a narrow model on an fp32 stream, no dropout
        dict(_ln(777, 1000, op="ln_bwd", residual="fp32", wfp32=True), name="ln_bwd_small_fp32"),
        # a training step's dropout of combine's output, joining the residual stream
        dict(op="dropout", T=16384, H=4096, x="bf16", residual=True, out="bf16", p=0.1, name="dropout_training"),
        # the branch's gradient from a small batch's fp32 stream gradient
        dict(op="dropout", T=100, H=1000, x="fp32", residual=False, out="bf16", p=0.25, name="dropout_small_bwd"),
        # a shared expert's second product for a few sequences: the weights are streamed once
        dict(_linear(16, 7168, 2048), name="linear_decode"),
        # a dense layer's projection of an odd batch, joined with the routed experts' sum
        dict(_linear(333, 4096, 4096, add=True), name="linear_ragged_add"),
        # a shared expert's gate and up projections over a prefill batch with the SwiGLU store
        dict(_linear(4096, 4096, 7168, swiglu=True), name="linear_prefill_swiglu"),
        # a training step's weight gradient: 16384 tokens contracted, added to the fp32 main gradient
        dict(_linear(1536, 4096, 16384, wscale="row", out="fp32", add=True, pow2=True), name="linear_wgrad_training"),
        # a weight's codes by squares, and their transpose for the data gradient, after an optimiser step
        dict(op="quantize", R=1536, C=4096, block="square", rows=True, pow2=False, name="quantize_weights"),
        # a training step's gradient rows, for the data gradient, and columns, for the weights'
        dict(op="quantize", R=16384, C=4096, block="rows", rows=True, pow2=True, name="quantize_training"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["ln", "ln", "ln_bwd", "ln_bwd", "dropout", "linear", "linear", "linear", "quantize"])
    if op in ("ln", "ln_bwd"):
        quant = "none" if op == "ln_bwd" else rng.choice(["none", "int8", "fp8", "fp8_pow2"])
        unit = {"none": 8, "int8": 16}.get(quant, 128)
        H = max(unit, _log(rng, 128, 8192) // unit * unit)
        return _ln(_log(rng, 1, 8192), H, op=op, residual=rng.choice(["none", "bf16", "bf16", "fp32"]),
                   wfp32=rng.random() < 0.4, bias=rng.random() < 0.8, p=rng.choice([0.0, 0.0, 0.1, 0.5]),
                   y=quant == "none" or rng.random() < 0.5, quant=quant)
    if op == "dropout":
        return dict(op=op, T=_log(rng, 1, 8192), H=8 * _log(rng, 1, 1024), x=rng.choice(["bf16", "bf16", "fp32"]),
                    residual=rng.random() < 0.5, out=rng.choice(["bf16", "fp32"]), p=rng.choice([0.05, 0.1, 0.25, 0.5]))
    if op == "quantize":
        return dict(op=op, R=_log(rng, 1, 8192), C=128 * _log(rng, 1, 56), block=rng.choice(["square", "rows"]),
                    rows=rng.random() < 0.7, pow2=rng.random() < 0.5)
    swiglu = rng.random() < 0.3
    N = 16 * _log(rng, 1, 400) if swiglu else _log(rng, 16, 6400)
    K = 128 * _log(rng, 1, 56)
    M = min(_log(rng, 1, 8192), max(1, 4096 * 4096 * 7168 // (N * K)))
    out = "bf16" if swiglu else rng.choice(["bf16", "bf16", "fp32"])
    return _linear(M, N, K, wscale=rng.choice(["block", "block", "row"]), out=out,
                   add=not swiglu and rng.random() < 0.4, swiglu=swiglu, pow2=rng.random() < 0.4)


def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _type(name):
    return torch.float32 if name == "fp32" else torch.bfloat16


def _empty(shape, dtype):
    return torch.empty(shape, dtype=dtype, device="cuda")


def prepare(case, seed):
    g = _generator(seed)
    op = case["op"]
    s = dict(case=case)
    if op in ("ln", "ln_bwd", "dropout"):
        # the generator's seed and this call's offset, as a training loop keeps them on the device
        s["rng"] = torch.randint(-2 ** 31, 2 ** 31, (4,), generator=g, device="cuda").to(torch.int32)
    if op in ("ln", "ln_bwd"):
        T, H = case["T"], case["H"]
        rt = _type(case["residual"])
        # a few channels carry large values and channels have means, as a residual stream's do
        spread, shift = torch.exp(_randn(g, H) * 0.5), _randn(g, H) * 0.3
        wt = torch.float32 if case["wfp32"] else torch.bfloat16
        s["weight"] = (1 + 0.2 * _randn(g, H)).to(wt)
        s["bias"] = (0.1 * _randn(g, H)).to(wt) if case["bias"] else None
        if op == "ln":
            s["x"] = (_randn(g, T, H) * spread).to(torch.bfloat16)
            s["residual"] = s["hidden"] = None
            if case["residual"] != "none":
                s["residual"] = (_randn(g, T, H) * spread * 2 + shift).to(rt)
            if case["residual"] != "none" or case["p"]:
                s["hidden"] = _empty((T, H), rt)
            s["y"] = _empty((T, H), torch.bfloat16) if case["y"] else None
            s["codes"] = s["scales"] = None
            if case["quant"] == "int8":
                s["codes"], s["scales"] = _empty((T, H), torch.int8), _empty((T,), torch.float32)
            elif case["quant"] != "none":
                s["codes"], s["scales"] = _empty((T, H), torch.float8_e4m3fn), _empty((T, H // 128), torch.float32)
        else:
            s["hidden"] = (_randn(g, T, H) * spread + shift).to(rt)
            s["gy"] = _randn(g, T, H).to(torch.bfloat16)
            s["gh"] = _randn(g, T, H).to(rt) if case["residual"] != "none" else None
            s["grad"] = _empty((T, H), rt)
            s["grad_x"] = _empty((T, H), torch.bfloat16) if case["p"] else None
            s["gweight"] = _empty((H,), torch.float32)
            s["gbias"] = _empty((H,), torch.float32) if case["bias"] else None
    elif op == "dropout":
        shape = (case["T"], case["H"])
        s["x"] = _randn(g, *shape).to(_type(case["x"]))
        s["residual"] = (_randn(g, *shape) * 2).to(_type(case["out"])) if case["residual"] else None
        s["out"] = _empty(shape, _type(case["out"]))
    elif op == "linear":
        M, N, K = case["M"], case["N"], case["K"]
        rows = _randn(g, M, K) * torch.exp(_randn(g, M, 1))
        s["x"], s["xs"] = _fp8(rows, 1, case["pow2"])
        w = _randn(g, N, K) * torch.exp(_randn(g, N, 1) * 0.3)
        s["w"], s["ws"] = _fp8(w, 128 if case["wscale"] == "block" else 1, case["pow2"])
        s["ws"] = s["ws"] * 2.0 ** -round(math.log2(math.sqrt(K)))   # results of the inputs' size
        shape = (M, N // 2 if case["swiglu"] else N)
        s["addend"] = _randn(g, *shape).to(_type(case["out"])) if case["add"] else None
        s["out"] = _empty(shape, _type(case["out"]))
    else:
        R, C = case["R"], case["C"]
        s["x"] = (_randn(g, R, C) * torch.exp(_randn(g, R, 1) * 0.5)).to(torch.bfloat16)
        Rp = (R + 127) // 128 * 128
        square = case["block"] == "square"
        s["codes"] = s["scales"] = None
        if case["rows"]:
            s["codes"] = _empty((R, C), torch.float8_e4m3fn)
            s["scales"] = _empty((Rp // 128 if square else R, C // 128), torch.float32)
        s["codes_t"] = _empty((C, Rp), torch.float8_e4m3fn)
        s["scales_t"] = _empty((C // 128 if square else C, Rp // 128), torch.float32)
    if own:
        import combine_ep_plan_amd as ep
        s["ep"] = ep
        if op == "ln_bwd":
            s["workspace"] = _empty((ep.ep_add_layernorm_bwd_workspace_bytes(case["T"], case["H"]) // 4,), torch.float32)
    return s


# ---------------------------------------------------------------------------
# plain forms


def _mul32(a, m):
    """High and low 32 bits of a 32-bit a times the 32-bit constant m, in int64."""
    upper, lower = (a >> 16) * m, (a & 0xFFFF) * m
    return (upper + (lower >> 16)) >> 16, (((upper & 0xFFFF) << 16) + lower) & 0xFFFFFFFF


def _keep(n, rng, p):
    """Which of n consecutive values stay: 16 bits each of Philox4x32-10 (Salmon et al., "Parallel random
    numbers: as easy as 1, 2, 3", 2011), a block of eight to a counter."""
    words = rng.long() & 0xFFFFFFFF
    k0, k1, o0, o1 = words[0], words[1], words[2], words[3]
    block = torch.arange((n + 7) // 8, device="cuda")
    c0, c1, c2, c3 = block & 0xFFFFFFFF, block >> 32, o0.expand_as(block), o1.expand_as(block)
    for _ in range(10):
        h0, l0 = _mul32(c0, 0xD2511F53)
        h1, l1 = _mul32(c2, 0xCD9E8D57)
        c0, c1, c2, c3 = h1 ^ c1 ^ k0, l1, h0 ^ c3 ^ k1, l0
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    u = torch.stack([c0 & 0xFFFF, c0 >> 16, c1 & 0xFFFF, c1 >> 16, c2 & 0xFFFF, c2 >> 16, c3 & 0xFFFF, c3 >> 16], 1)
    return u.view(-1)[:n] < _threshold(p)


def _threshold(p):
    return int(math.floor((1 - p) * 65536 + 0.5))


def _scale(p):
    """1 / (the probability of staying), as the 32-bit number it is multiplied by."""
    return float(np.float32(65536.0 / _threshold(p)))


def _dropped(x, rng, p):
    """In 64 bits, so that the sum with the stream is rounded once."""
    if not p:
        return x.double()
    keep = _keep(x.numel(), rng, p).view(x.shape)
    return torch.where(keep, x.double() * _scale(p), 0)


def _joined(x, rng, p, residual, dtype):
    h = _dropped(x, rng, p)
    if residual is not None:
        h = h + residual.double()
    return h.float().to(dtype)


def _amax_scale(amax, most, pow2=False):
    scale = torch.where(amax > 0, amax / most, 1)
    if pow2:
        m, e = torch.frexp(scale.double())
        up = torch.ldexp(torch.ones_like(m), torch.where(m > 0.5, e, e - 1)).clamp(min=2.0 ** -126)
        scale = torch.where(amax > 0, up.float(), 1)
    return scale


def _fp8(x, rows, pow2):
    """Codes and scales of x by blocks of rows x 128 (the last rows may be fewer)."""
    R, C = x.shape
    Rp = (R + rows - 1) // rows * rows
    v = torch.cat([x, x.new_zeros(Rp - R, C)]) if Rp > R else x
    v = v.float().view(Rp // rows, rows, C // 128, 128)
    scale = _amax_scale(v.abs().amax((1, 3), keepdim=True), 448, pow2)
    codes = (v / scale).clamp(-448, 448).to(torch.float8_e4m3fn)
    return codes.view(Rp, C)[:R].contiguous(), scale.view(Rp // rows, C // 128)


def _int8(y):
    scale = _amax_scale(y.abs().amax(1, keepdim=True), 127)
    # the nearest integer to the exact quotient (64 bits tell its ties from their neighbours)
    return torch.round(y.double() / scale.double()).clamp(-127, 127).to(torch.int8), scale.squeeze(1)


def _centred(h):
    """h - mean and 1 / sqrt(variance + eps): the long sums in 64 bits, each rounded once."""
    d = h.double() - h.double().mean(1, keepdim=True)
    return d.float(), (1 / torch.sqrt(d.square().mean(1, keepdim=True) + EPS)).float()


def _run_ln(s):
    case = s["case"]
    h, out = s["x"], []
    if s["hidden"] is not None:
        h = _joined(h, s["rng"], case["p"], s["residual"], s["hidden"].dtype)
        out.append(h)
    d, r = _centred(h)
    y = d * r
    if s["bias"] is None:
        y = y * s["weight"].float()
    else:
        y = (y.double() * s["weight"].double() + s["bias"].double()).float()
    if case["y"]:
        out.append(y.to(torch.bfloat16))
    if case["quant"] == "int8":
        out += _int8(y)
    elif case["quant"] != "none":
        out += _fp8(y, 1, case["quant"] == "fp8_pow2")
    return out


def _run_ln_bwd(s):
    gy = s["gy"].float()
    d, r = _centred(s["hidden"])
    n = d * r
    g = gy * s["weight"].float()
    mg = g.double().mean(1, keepdim=True).float()
    mn = (g.double() * n.double()).mean(1, keepdim=True).float()
    grad = r * (g - mg - n * mn)
    if s["gh"] is not None:
        grad = grad + s["gh"].float()
    out = [grad.to(s["grad"].dtype)]
    if s["grad_x"] is not None:
        out.append(_dropped(grad, s["rng"], s["case"]["p"]).float().to(torch.bfloat16))
    out.append((gy * n).sum(0))
    return out + [gy.sum(0)] if s["gbias"] is not None else out


def _run_dropout(s):
    return _joined(s["x"], s["rng"], s["case"]["p"], s["residual"], s["out"].dtype)


def _values(codes, scales, rows):
    R, C = codes.shape
    s = scales if rows == 1 else scales.repeat_interleave(rows, 0)[:R]
    return (codes.float().view(R, C // 128, 128) * s.unsqueeze(2)).view(R, C)


def _run_linear(s):
    case = s["case"]
    x = _values(s["x"], s["xs"], 1)
    w = _values(s["w"], s["ws"], 128 if case["wscale"] == "block" else 1)
    h = torch.mm(x, w.t())
    if case["swiglu"]:
        gate, up = h[:, 0::2], h[:, 1::2]
        h = gate / (1 + torch.exp(-gate)) * up
    if s["addend"] is not None:
        h = h + s["addend"].float()
    return h.to(s["out"].dtype)


def _run_quantize(s):
    case, x = s["case"], s["x"]
    R, C = x.shape
    Rp = s["codes_t"].shape[1]
    rows = 128 if case["block"] == "square" else 1
    t = torch.cat([x, x.new_zeros(Rp - R, C)]) if Rp > R else x
    out = list(_fp8(x, rows, case["pow2"])) if case["rows"] else []
    return out + list(_fp8(t.t().contiguous(), rows, case["pow2"]))


_PLAIN = dict(ln=_run_ln, ln_bwd=_run_ln_bwd, dropout=_run_dropout, linear=_run_linear, quantize=_run_quantize)


def run(s):
    return _own(s) if own else _PLAIN[s["case"]["op"]](s)


# ---------------------------------------------------------------------------
# the library's calls


def _own(s):
    ep, case = s["ep"], s["case"]
    op = case["op"]
    if op == "ln":
        ep.ep_add_layernorm(s["x"], s["residual"], s["weight"], s["bias"], s["hidden"], s["y"], s["codes"],
                            s["scales"], eps=EPS, quant=case["quant"], dropout=case["p"],
                            rng=s["rng"] if case["p"] else None)
        return [s[n] for n in ("hidden", "y", "codes", "scales") if s[n] is not None]
    if op == "ln_bwd":
        ep.ep_add_layernorm_bwd(s["hidden"], s["weight"], s["gy"], s["gh"], s["grad"], s["grad_x"], s["gweight"],
                                s["gbias"], s["workspace"], eps=EPS, dropout=case["p"],
                                rng=s["rng"] if case["p"] else None)
        return [s[n] for n in ("grad", "grad_x", "gweight", "gbias") if s[n] is not None]
    if op == "dropout":
        ep.ep_dropout(s["x"], s["residual"], s["out"], case["p"], s["rng"])
        return s["out"]
    if op == "linear":
        ep.ep_linear_fp8(s["x"], s["xs"], s["w"], s["ws"], s["addend"], s["out"], swiglu=case["swiglu"],
                         pow2=case["pow2"])
        return s["out"]
    ep.ep_quantize_fp8_2d(s["x"], s["codes"], s["scales"], s["codes_t"], s["scales_t"], block=case["block"],
                          pow2=case["pow2"])
    return [s[n] for n in ("codes", "scales", "codes_t", "scales_t") if s[n] is not None]


# ---------------------------------------------------------------------------
# what one pass cannot do without


def work(case):
    op = case["op"]
    if op in ("ln", "ln_bwd", "dropout"):
        n = case["T"] * case["H"]
        philox = 12 * n if case["p"] else 0
        if op == "dropout":
            xb, ob = (4 if case[k] == "fp32" else 2 for k in ("x", "out"))
            return {"bytes": n * (xb + ob + ob * case["residual"]), "flops": 2 * n + philox}
        rb = 4 if case["residual"] == "fp32" else 2
        has = case["residual"] != "none"
        if op == "ln":
            b = 2 * n + rb * n * has + rb * n * (has or case["p"] > 0) + 2 * n * case["y"] + n * (case["quant"] != "none")
            return {"bytes": b, "flops": 12 * n + philox}
        return {"bytes": rb * n + 2 * n + rb * n * has + rb * n + 2 * n * (case["p"] > 0), "flops": 18 * n + philox}
    if op == "quantize":
        n = case["R"] * case["C"]
        return {"bytes": 2 * n + n * case["rows"] + n, "flops": 4 * n}
    M, N, K = case["M"], case["N"], case["K"]
    ob = (4 if case["out"] == "fp32" else 2) * M * (N // 2 if case["swiglu"] else N)
    scales = 4 * (K // 128) * (M + (N if case["wscale"] == "row" else (N + 127) // 128))
    return {"bytes": (M + N) * K + scales + ob * (1 + case["add"]), "flops": 2 * M * N * K}


# ---------------------------------------------------------------------------
# the definitions in 64 bits


def _np(t):
    return None if t is None else t.detach().double().cpu().numpy()


def _exact_factor(s, shape):
    """0 or 1 / (the probability of staying) of each value."""
    p = s["case"]["p"]
    if not p:
        return np.ones(shape)
    key = s["rng"].cpu().numpy().view(np.uint32).astype(np.uint64)
    n = int(np.prod(shape))
    mask = np.uint64(0xFFFFFFFF)
    b = np.arange((n + 7) // 8, dtype=np.uint64)
    ctr = [b & mask, b >> np.uint64(32), np.full_like(b, key[2]), np.full_like(b, key[3])]
    k = [key[0], key[1]]
    for r in range(10):
        a, c = ctr[0] * np.uint64(0xD2511F53), ctr[2] * np.uint64(0xCD9E8D57)
        ctr = [(c >> np.uint64(32)) ^ ctr[1] ^ k[0], c & mask, (a >> np.uint64(32)) ^ ctr[3] ^ k[1], a & mask]
        k = [(k[0] + np.uint64(0x9E3779B9)) & mask, (k[1] + np.uint64(0xBB67AE85)) & mask]
    u = np.stack(ctr, 1).astype(np.uint32).view(np.uint16).reshape(-1)[:n]
    stay = np.floor((1 - p) * 65536 + 0.5)
    return np.where(u < stay, 65536 / stay, 0.0).reshape(shape)


def _rounded(h, dtype):
    """What the stream holds of h."""
    return torch.from_numpy(h).to(dtype).double().numpy()


def _exact_ln(case, s):
    h = _np(s["x"])
    out = []
    if s["hidden"] is not None:
        h = h * _exact_factor(s, h.shape)
        if s["residual"] is not None:
            h += _np(s["residual"])
        out.append(h)
        h = _rounded(h, s["hidden"].dtype)   # that is what is normalised
    mu = h.mean(1, keepdims=True)
    y = (h - mu) / np.sqrt(h.var(1, keepdims=True) + EPS) * _np(s["weight"])
    if s["bias"] is not None:
        y += _np(s["bias"])
    if case["y"]:
        out.append(y)
    if case["quant"] == "int8":
        a = np.abs(y).max(1)
        scale = np.where(a > 0, a / 127.0, 1.0)
        out += [np.clip(np.rint(y / scale[:, None]), -127, 127).astype(np.int8), scale]
    elif case["quant"] != "none":
        out += _exact_fp8(y, 1, case["quant"] == "fp8_pow2")
    return out


def _exact_fp8(v, rows, pow2):
    """Quotients by the scales (what the codes round) and the scales."""
    R, C = v.shape
    Rp = -(-R // rows) * rows
    b = np.zeros((Rp, C))
    b[:R] = np.abs(v)
    a = b.reshape(Rp // rows, rows, C // 128, 128).max((1, 3))
    scale = np.where(a > 0, a / 448.0, 1.0)
    if pow2:
        scale = np.where(a > 0, np.exp2(np.ceil(np.log2(scale))), 1.0)
    return [v / np.repeat(np.repeat(scale, rows, 0)[:R], 128, 1), scale]


def _exact_ln_bwd(case, s):
    h, gy = _np(s["hidden"]), _np(s["gy"])
    x = h - h.mean(1, keepdims=True)
    r = 1.0 / np.sqrt((x * x).mean(1, keepdims=True) + EPS)
    g = gy * _np(s["weight"])
    grad = (g - g.mean(1, keepdims=True)) * r - x * r ** 3 * (g * x).mean(1, keepdims=True)
    if s["gh"] is not None:
        grad = grad + _np(s["gh"])
    out = [grad]
    if s["grad_x"] is not None:
        out.append(grad * _exact_factor(s, grad.shape))
    out.append((gy * x * r).sum(0))
    return out + [gy.sum(0)] if s["gbias"] is not None else out


def _exact_dropout(case, s):
    v = _np(s["x"]) * _exact_factor(s, tuple(s["x"].shape))
    return v if s["residual"] is None else v + _np(s["residual"])


def _exact_linear(case, s):
    K = case["K"]
    out = torch.zeros(s["x"].shape[0], case["N"], dtype=torch.float64, device="cuda")
    for b in range(K // 128):   # block by block, as the formula has it
        part = s["x"][:, 128 * b:128 * b + 128].double() @ s["w"][:, 128 * b:128 * b + 128].double().t().contiguous()
        sw = s["ws"][:, b].double()
        if case["wscale"] == "block":
            sw = sw.repeat_interleave(128)[:case["N"]]
        out += part * s["xs"][:, b].double()[:, None] * sw[None]
    if case["swiglu"]:
        h = out.view(out.shape[0], -1, 2)
        out = h[..., 0] / (1.0 + torch.exp(-h[..., 0])) * h[..., 1]
    return out if s["addend"] is None else out + s["addend"].double()


def _exact_quantize(case, s):
    x = _np(s["x"])
    rows = 128 if case["block"] == "square" else 1
    t = np.zeros((x.shape[1], s["codes_t"].shape[1]))
    t[:, :x.shape[0]] = x.T
    return (_exact_fp8(x, rows, case["pow2"]) if case["rows"] else []) + _exact_fp8(t, rows, case["pow2"])


_EXACT = dict(ln=_exact_ln, ln_bwd=_exact_ln_bwd, dropout=_exact_dropout, linear=_exact_linear,
              quantize=_exact_quantize)


def exact(case, seed):
    global own
    was, own = own, False   # the inputs alone: nothing of the library is made
    try:
        return _EXACT[case["op"]](case, prepare(case, seed))
    finally:
        own = was
