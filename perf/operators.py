"""Measured operators: scored routing, residual add + RMS norm with 8-bit
outputs, 8-bit rows (quantiser and dispatch), and the INT8 grouped GEMM of
the experts.

``run`` computes them as elementary torch operations, or with ``own`` by the
library's entry points.  Both take the inputs ``prepare`` makes; a state
holds its inputs, its output buffers and (``own``) the planned handle a
program keeps."""

import math

import numpy as np
import torch

own = False

# The shapes are this repository's workloads: decode (T 128, H 7168, E 256,
# top-8, LL), prefill (T 4096, H 7168, E 256, top-8, HT, skewed), training
# (T 16384, H 4096, E 128, top-8).
EPS = 1e-6


def _route(T, E, k, **kw):
    c = dict(op="route", T=T, E=E, k=k, score="sigmoid", bias=True, groups=1, kept=1, top2=False,
             renorm=True, scale=1.0, bf16=False, scores=False, masked=0.0)
    c.update(kw)
    return c


def _norm(T, H, **kw):
    c = dict(op="norm", T=T, H=H, residual="bf16", wfp32=False, y=True, quant="none")
    c.update(kw)
    return c


def listed():
    return [
        # the router of a decode step: sigmoid scores, balance bias, 4 of 8 expert groups
        dict(_route(128, 256, 8, groups=8, kept=4, top2=True, scale=2.5), name="route_decode"),
        # the router of a prefill batch, the same rule
        dict(_route(4096, 256, 8, groups=8, kept=4, top2=True, scale=2.5), name="route_prefill"),
        # the router's backward in a training step, softmax over all experts, with the gradient a
        # balance loss puts on the scores
        dict(_route(16384, 128, 8, op="route_bwd", score="softmax", bias=False, renorm=False, scores=True),
             name="route_bwd_training"),
        # a decode step's norm: residual added, bf16 rows for the router and INT8 rows for the experts
        dict(_norm(128, 7168, quant="int8"), name="norm_decode_int8"),
        # a prefill batch's norm with FP8 rows
        dict(_norm(4096, 7168, quant="fp8"), name="norm_prefill_fp8"),
        # the norm's backward in a training step, the residual stream's gradient joining
        dict(_norm(16384, 4096, op="norm_bwd"), name="norm_bwd_training"),
        # the activation between an expert FFN's two products: a decode step's rows, a prefill batch's
        dict(op="quantize", rows=1024, K=2048, name="quantize_decode"),
        dict(op="quantize", rows=32768, K=2048, name="quantize_prefill"),
        # INT8 rows to their experts: a decode step (LL, 128 rows an expert), a prefill batch (HT)
        dict(op="dispatch", T=128, H=7168, E=256, k=8, layout="ll", cap=128, skew=0.0, fmt="int8",
             name="dispatch_decode"),
        dict(op="dispatch", T=4096, H=7168, E=256, k=8, layout="ht", cap=0, skew=1.1, fmt="int8",
             name="dispatch_prefill"),
        # the experts' INT8 products: a decode step, which streams every expert's weights ...
        dict(op="gemm", T=128, E=256, k=8, K=7168, N=2048, layout="ll", cap=128, skew=0.0, swiglu=False,
             name="gemm_decode"),
        # ... and a prefill batch's gate and up projections with the SwiGLU store
        dict(op="gemm", T=4096, E=256, k=8, K=7168, N=4096, layout="ht", cap=0, skew=1.1, swiglu=True,
             name="gemm_prefill_swiglu"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "route", "route_bwd", "norm", "norm", "norm_bwd", "quantize", "dispatch", "gemm"])
    if op in ("route", "route_bwd"):
        E = rng.choice([8, 60, 64, 100, 128, 160, 256, 384, 512])
        groups = rng.choice([g for g in (1, 1, 2, 4, 8, 10, 16) if E % g == 0])
        c = _route(_log(rng, 1, 16384), E, rng.choice([1, 2, 4, 6, 8]), op=op,
                   score=rng.choice(["softmax", "sigmoid"]), bias=rng.random() < 0.6, groups=groups,
                   kept=rng.randint(1, groups), top2=rng.random() < 0.5, renorm=rng.random() < 0.6,
                   scale=rng.choice([1.0, 2.5]), bf16=rng.random() < 0.3, scores=rng.random() < 0.4,
                   masked=rng.choice([0.0, 0.0, 0.05]))
        return c
    if op in ("norm", "norm_bwd"):
        quant = "none" if op == "norm_bwd" else rng.choice(["none", "int8", "fp8", "fp8_pow2"])
        unit = {"none": 8, "int8": 16}.get(quant, 128)
        H = max(unit, _log(rng, 128, 8192) // unit * unit)
        residual = rng.choice(["none", "bf16", "bf16", "fp32"])
        return _norm(_log(rng, 1, 8192), H, op=op, residual=residual, wfp32=rng.random() < 0.4,
                     y=quant == "none" or rng.random() < 0.5, quant=quant)
    if op == "quantize":
        return dict(op=op, rows=_log(rng, 1, 32768), K=16 * _log(rng, 1, 448))
    E = rng.choice([8, 32, 128, 256])
    k = rng.choice([1, 2, 4, 6, 8])
    layout = rng.choice(["ll", "ht"])
    T = _log(rng, 1, 256 if layout == "ll" else 4096)
    skew = rng.choice([0.0, 1.1])
    cap = T if layout == "ll" else 0
    if op == "dispatch":
        return dict(op=op, T=T, H=128 * rng.randint(1, 56), E=E, k=k, layout=layout, cap=cap, skew=skew,
                    fmt=rng.choice(["int8", "fp8"]))
    return dict(op=op, T=T, E=E, k=k, K=64 * _log(rng, 1, 112), N=16 * _log(rng, 1, 256), layout=layout,
                cap=cap, skew=skew, swiglu=rng.random() < 0.5)


def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _routing(case, g):
    """Top-k ids of a router with a popular head of experts (skew 0: none), each expert's entry count
    and each entry's receive row."""
    T, E, k = case["T"], case["E"], case["k"]
    logits = _randn(g, T, E) - case["skew"] * torch.log(torch.arange(1, E + 1, device="cuda").float())
    idx = torch.topk(logits, k, dim=1).indices.to(torch.int32)
    flat = idx.reshape(-1).long()
    counts = torch.bincount(flat, minlength=E)
    order = torch.sort(flat, stable=True).indices
    at = torch.empty_like(flat)
    at[order] = torch.arange(T * k, device="cuda")
    if case["layout"] == "ll":
        at = at - (torch.cumsum(counts, 0) - counts)[flat] + flat * case["cap"]
    rows = E * case["cap"] if case["layout"] == "ll" else T * k
    return idx, counts, at, rows


def _int8_rows(g, rows, K):
    """Codes and scales as a quantiser leaves them: bell-shaped, the row's largest at 127."""
    codes = torch.empty(rows, K, dtype=torch.int8, device="cuda")
    step = max(1, (1 << 28) // K)
    for r in range(0, rows, step):
        x = _randn(g, min(step, rows - r), K)
        codes[r:r + step] = torch.round(x * 32).clamp_(-127, 127).to(torch.int8)
    return codes, torch.rand(rows, generator=g, device="cuda") * 0.03 + 0.005


def prepare(case, seed):
    g = _generator(seed)
    op = case["op"]
    s = dict(case=case)
    if op in ("route", "route_bwd"):
        T, E, k = case["T"], case["E"], case["k"]
        l = _randn(g, T, E) * 1.5
        if case["masked"]:
            # experts a request may not use; now and then all of them
            l[torch.rand(T, E, generator=g, device="cuda") < case["masked"]] = -math.inf
            l[torch.rand(T, generator=g, device="cuda") < case["masked"]] = -math.inf
        s["logits"] = l.to(torch.bfloat16) if case["bf16"] else l
        s["bias"] = _randn(g, E) * 0.1 if case["bias"] else None
        s["idx"] = torch.empty(T, k, dtype=torch.int32, device="cuda")
        s["w"] = torch.empty(T, k, device="cuda")
        s["scores"] = torch.empty(T, E, device="cuda") if case["scores"] else None
        if op == "route_bwd":
            s["idx"] = _choose(case, s["logits"], s["bias"])[0].to(torch.int32)
            s["gw"] = _randn(g, T, k)
            s["gs"] = _randn(g, T, E) * 0.01 if case["scores"] else None
            s["gl"] = torch.empty_like(s["logits"])
    elif op in ("norm", "norm_bwd"):
        T, H = case["T"], case["H"]
        rt = torch.float32 if case["residual"] == "fp32" else torch.bfloat16
        # a few channels carry large values, as a residual stream's do
        spread = torch.exp(_randn(g, H) * 0.5)
        s["weight"] = 1 + 0.2 * _randn(g, H)
        if not case["wfp32"]:
            s["weight"] = s["weight"].to(torch.bfloat16)
        if op == "norm":
            s["x"] = (_randn(g, T, H) * spread).to(torch.bfloat16)
            if case["residual"] != "none":
                s["residual"] = (_randn(g, T, H) * spread * 2).to(rt)
                s["hidden"] = torch.empty_like(s["residual"])
            s["y"] = torch.empty(T, H, dtype=torch.bfloat16, device="cuda") if case["y"] else None
            if case["quant"] == "int8":
                s["codes"] = torch.empty(T, H, dtype=torch.int8, device="cuda")
                s["scales"] = torch.empty(T, device="cuda")
            elif case["quant"] != "none":
                s["codes"] = torch.empty(T, H, dtype=torch.float8_e4m3fn, device="cuda")
                s["scales"] = torch.empty(T, H // 128, device="cuda")
        else:
            s["hidden"] = (_randn(g, T, H) * spread).to(rt)
            s["gy"] = _randn(g, T, H).to(torch.bfloat16)
            s["gh"] = _randn(g, T, H).to(rt) if case["residual"] != "none" else None
            s["gx"] = torch.empty(T, H, dtype=rt, device="cuda")
            s["gweight"] = torch.empty(H, device="cuda")
    elif op == "quantize":
        s["x"] = (_randn(g, case["rows"], case["K"]) * torch.exp(_randn(g, case["rows"], 1))).to(torch.bfloat16)
        s["codes"] = torch.empty(case["rows"], case["K"], dtype=torch.int8, device="cuda")
        s["scales"] = torch.empty(case["rows"], device="cuda")
    else:
        s["idx"], counts, s["dst"], rows = _routing(case, g)
        s["counts"] = counts.tolist()
        if op == "dispatch":
            T, H = case["T"], case["H"]
            s["codes"], s["scales"] = _int8_rows(g, T, H)
            if case["fmt"] == "fp8":
                s["codes"] = (_randn(g, T, H) * 100).clamp(-448, 448).to(torch.float8_e4m3fn)
                s["scales"] = torch.rand(T, H // 128, generator=g, device="cuda") + 0.1
            s["recv"] = torch.zeros(rows, H, dtype=torch.int8, device="cuda").view(s["codes"].dtype)
            s["recv_scales"] = torch.zeros((rows,) + tuple(s["scales"].shape[1:]), device="cuda")
        else:
            E, N, K = case["E"], case["N"], case["K"]
            s["x"], s["xs"] = _int8_rows(g, rows, K)
            w, ws = _int8_rows(g, E * N, K)
            s["w"], s["ws"] = w.view(E, N, K), ws.view(E, N) * (0.2 / math.sqrt(K))
            s["out"] = torch.zeros(rows, N // 2 if case["swiglu"] else N, dtype=torch.bfloat16, device="cuda")
    if own:
        _keep(case, s)
    return s


def _keep(case, s):
    """What a program of the library keeps from call to call: groups, planned handles, workspaces."""
    import combine_ep_plan_amd as ep
    op = case["op"]
    s["ep"] = ep
    if op in ("route", "route_bwd"):
        s["group"] = ep.Group(case["E"], 1, 8, case["k"], case["T"], "ht")
        s["handle"] = ep.Handle(s["group"], case["T"])
        s["rule"] = ep.RouteRule(score=case["score"], num_groups=case["groups"], kept_groups=case["kept"],
                                 group_score="top2" if case["top2"] else "max", renormalise=case["renorm"],
                                 scale=case["scale"])
    elif op == "norm_bwd":
        s["workspace"] = torch.empty(ep.ep_add_rmsnorm_bwd_workspace_bytes(case["T"], case["H"]) // 4,
                                     device="cuda")
    elif op in ("dispatch", "gemm"):
        s["group"] = ep.Group(case["E"], 1, case.get("H", 128), case["k"], case["T"], case["layout"],
                              capacity=case["cap"])
        s["handle"] = ep.Handle(s["group"], case["T"]).plan(s["idx"])


# ---------------------------------------------------------------------------
# plain forms


def _choose(case, logits, bias):
    """Ids, the experts' scores and the clean logits (masked: -inf), in 64 bits: two experts at a border
    differ by less than 32 bits tell."""
    l = logits.double()
    l = torch.where(torch.isnan(l), -math.inf, l).clamp(max=torch.finfo(torch.float32).max)
    live = l > -math.inf
    if case["score"] == "sigmoid":
        score = 1 / (1 + torch.exp(-l))
    else:
        top = torch.where(live, l, torch.finfo(torch.float32).min).amax(1, keepdim=True)
        e = torch.where(live, torch.exp(l - top), 0)
        score = e / e.sum(1, keepdim=True).clamp(min=1e-300)
    # without a bias or sums over a group, the order of the scores is that of the logits
    by_logit = bias is None and not (case["groups"] > 1 and case["top2"])
    choice = l if by_logit else score if bias is None else score + bias.double()
    choice = torch.where(live, choice, -math.inf)
    if case["groups"] > 1:
        per = choice.view(choice.shape[0], case["groups"], -1)
        best = torch.sort(per, dim=2, descending=True).values
        value = best[..., 0]
        if case["top2"] and per.shape[2] > 1:
            second = best[..., 1]
            value = torch.where(second > -math.inf, value + second, value)
        order = torch.sort(value, dim=1, descending=True, stable=True).indices
        keep = torch.zeros_like(value, dtype=torch.bool)
        keep.scatter_(1, order[:, :case["kept"]], True)
        choice = torch.where(keep.unsqueeze(2), per, -math.inf).view_as(choice)
    got = torch.sort(choice, dim=1, descending=True, stable=True)
    k = case["k"]
    idx, value = got.indices[:, :k], got.values[:, :k]
    idx = torch.where(value > -math.inf, idx, -1)
    if idx.shape[1] < k:
        idx = torch.cat([idx, idx.new_full((idx.shape[0], k - idx.shape[1]), -1)], 1)
    return idx, score, l


def _weights(case, idx, score, l):
    chosen = idx >= 0
    at = idx.clamp(min=0)
    if not case["renorm"]:
        return torch.where(chosen, torch.gather(score, 1, at), 0) * case["scale"], chosen, at
    u = torch.gather(l, 1, at)
    if case["score"] == "sigmoid":   # log of the score, so that no sum is ever zero
        u = u.clamp(max=0) - torch.log1p(torch.exp(-u.abs()))
    u = torch.where(chosen, u, -math.inf)
    e = torch.where(chosen, torch.exp(u - u.amax(1, keepdim=True)), 0)
    return e / e.sum(1, keepdim=True).clamp(min=1e-300) * case["scale"], chosen, at


def _run_route(s):
    case = s["case"]
    idx, score, l = _choose(case, s["logits"], s["bias"])
    w, _, _ = _weights(case, idx, score, l)
    out = [idx.to(torch.int32), w.float()]
    return out + [score.float()] if case["scores"] else out


def _run_route_bwd(s):
    case = s["case"]
    l = s["logits"].float()
    live = l > -math.inf
    if case["score"] == "sigmoid":
        score, slope = 1 / (1 + torch.exp(-l)), 1 / (1 + torch.exp(l))
    else:
        top = torch.where(live, l, torch.finfo(torch.float32).min).amax(1, keepdim=True)
        e = torch.where(live, torch.exp(l - top), 0)
        score = e / e.sum(1, keepdim=True).clamp(min=1e-30)
    w, chosen, at = _weights(dict(case, scale=1.0), s["idx"].long(), score, l)
    gw = torch.where(chosen, s["gw"], 0) * case["scale"]
    gl = torch.zeros_like(l)
    if case["renorm"]:   # through the shares w of the chosen: the logits' softmax, or the scores'
        part = w * (gw - (gw * w).sum(1, keepdim=True))
        if case["score"] == "sigmoid":
            part = part * torch.gather(slope, 1, at)
        gl.scatter_add_(1, at, torch.where(chosen, part, 0))
    gs = torch.zeros_like(l) if s["gs"] is None else s["gs"].clone()
    if not case["renorm"]:
        gs.scatter_add_(1, at, gw)
    if s["gs"] is not None or not case["renorm"]:
        if case["score"] == "sigmoid":
            gl = gl + gs * score * slope
        else:
            gl = gl + score * (gs - (gs * score).sum(1, keepdim=True))
    return torch.where(live, gl, 0).to(s["logits"].dtype)


def _rstd(h):
    """1 / sqrt(mean h^2 + eps): the long sum in 64 bits, rounded once."""
    return (1 / torch.sqrt(h.double().square().mean(1, keepdim=True) + EPS)).float()


def _int8(y, amax):
    scale = torch.where(amax > 0, amax / 127, 1)
    # the nearest integer to the exact quotient (64 bits tell its ties from their neighbours)
    return torch.round(y.double() / scale.double()).clamp(-127, 127).to(torch.int8), scale.squeeze(1)


def _fp8(y, pow2):
    T, H = y.shape
    b = y.view(T, H // 128, 128)
    amax = b.abs().amax(2, keepdim=True)
    scale = torch.where(amax > 0, amax / 448, 1)
    if pow2:
        m, e = torch.frexp(scale.double())
        up = torch.ldexp(torch.ones_like(m), torch.where(m > 0.5, e, e - 1)).clamp(min=2.0 ** -126)
        scale = torch.where(amax > 0, up.float(), 1)
    return (b / scale).clamp(-448, 448).to(torch.float8_e4m3fn).view(T, H), scale.squeeze(2)


def _run_norm(s):
    case = s["case"]
    h = s["x"]
    out = []
    if case["residual"] != "none":
        h = (h.float() + s["residual"].float()).to(s["residual"].dtype)
        out.append(h)
    y = h.float() * s["weight"].float() * _rstd(h)
    if case["y"]:
        out.append(y.to(torch.bfloat16))
    if case["quant"] == "int8":
        out += _int8(y, y.abs().amax(1, keepdim=True))
    elif case["quant"] != "none":
        out += _fp8(y, case["quant"] == "fp8_pow2")
    return out


def _run_norm_bwd(s):
    h, gy, w = s["hidden"].float(), s["gy"].float(), s["weight"].float()
    r = _rstd(s["hidden"])
    n = h * r
    g = gy * w
    gx = r * (g - n * (g * n).mean(1, keepdim=True))
    if s["gh"] is not None:
        gx = gx + s["gh"].float()
    return [gx.to(s["hidden"].dtype), (gy * n).sum(0)]


def _run_quantize(s):
    y = s["x"].float()
    return list(_int8(y, y.abs().amax(1, keepdim=True)))


def _run_dispatch(s):
    token = torch.arange(s["dst"].numel(), device="cuda") // s["case"]["k"]
    recv = torch.zeros_like(s["recv"].view(torch.int8))
    recv[s["dst"]] = s["codes"].view(torch.int8)[token]
    scales = torch.zeros_like(s["recv_scales"])
    scales[s["dst"]] = s["scales"][token]
    return [recv.view(s["codes"].dtype), scales]


def _groups(case, counts):
    """(expert, first row, rows) of every expert that has rows."""
    out, row = [], 0
    for e, n in enumerate(counts):
        if n:
            out.append((e, e * case["cap"] if case["layout"] == "ll" else row, n))
        row += n
    return out


def _run_gemm(s):
    case = s["case"]
    out = torch.zeros_like(s["out"])
    for e, r, n in _groups(case, s["counts"]):
        h = torch.mm(s["x"][r:r + n].float(), s["w"][e].float().t())
        h = h * (s["xs"][r:r + n].unsqueeze(1) * s["ws"][e])
        if case["swiglu"]:
            gate, up = h[:, 0::2], h[:, 1::2]
            h = gate / (1 + torch.exp(-gate)) * up
        out[r:r + n] = h.to(torch.bfloat16)
    return out


_PLAIN = dict(route=_run_route, route_bwd=_run_route_bwd, norm=_run_norm, norm_bwd=_run_norm_bwd,
              quantize=_run_quantize, dispatch=_run_dispatch, gemm=_run_gemm)


def run(s):
    return _own(s) if own else _PLAIN[s["case"]["op"]](s)


# ---------------------------------------------------------------------------
# the library's calls


def _own(s):
    ep, case = s["ep"] if "ep" in s else None, s["case"]
    op = case["op"]
    if op == "route":
        ep.ep_route_scored(s["handle"].ptr, s["rule"], s["logits"], s["bias"], s["idx"], s["w"], s["scores"])
        return [s["idx"], s["w"]] + ([s["scores"]] if case["scores"] else [])
    if op == "route_bwd":
        ep.ep_route_scored_bwd(s["handle"].ptr, s["rule"], s["logits"], s["idx"], s["gw"], s["gs"], s["gl"])
        return s["gl"]
    if op == "norm":
        ep.ep_add_rmsnorm(s["x"], s.get("residual"), s["weight"], s.get("hidden"), s["y"], s.get("codes"),
                          s.get("scales"), eps=EPS, quant=case["quant"])
        return [s[n] for n in ("hidden", "y", "codes", "scales") if s.get(n) is not None]
    if op == "norm_bwd":
        ep.ep_add_rmsnorm_bwd(s["hidden"], s["weight"], s["gy"], s["gh"], s["gx"], s["gweight"],
                              s["workspace"], eps=EPS)
        return [s["gx"], s["gweight"]]
    if op == "quantize":
        ep.ep_quantize_int8(s["x"], s["codes"], s["scales"])
        return [s["codes"], s["scales"]]
    if op == "dispatch":
        ep.ep_dispatch_quantized(s["handle"].ptr, s["codes"], s["scales"], None, s["recv"], s["recv_scales"])
        return [s["recv"], s["recv_scales"]]
    ep.ep_expert_gemm_int8(s["handle"].ptr, s["x"], s["xs"], s["w"], s["ws"], None, None, s["out"],
                           swiglu=case["swiglu"])
    return s["out"]


# ---------------------------------------------------------------------------
# what one pass cannot do without


def _experts_used(case):
    """Experts that get an entry, on average over even routing."""
    return case["E"] * (1 - (1 - 1 / case["E"]) ** (case["T"] * case["k"]))


def work(case):
    op = case["op"]
    if op in ("route", "route_bwd"):
        T, E, k = case["T"], case["E"], case["k"]
        cell = T * E * (2 if case["bf16"] else 4)
        scores = 4 * T * E if case["scores"] else 0
        if op == "route":
            return {"bytes": cell + 4 * E * case["bias"] + 8 * T * k + scores, "flops": 12 * T * E}
        dense = case["scores"] or (case["score"] == "softmax" and not case["renorm"])
        read = cell if dense else T * k * 4
        return {"bytes": read + cell + 8 * T * k + scores, "flops": 12 * T * E if dense else 12 * T * k}
    if op in ("norm", "norm_bwd"):
        n = case["T"] * case["H"]
        rb = 4 if case["residual"] == "fp32" else 2
        has = case["residual"] != "none"
        if op == "norm":
            b = 2 * n + 2 * rb * n * has + 2 * n * case["y"] + n * (case["quant"] != "none")
            return {"bytes": b, "flops": 10 * n}
        return {"bytes": rb * n + 2 * n + rb * n * has + rb * n, "flops": 14 * n}
    if op == "quantize":
        n = case["rows"] * case["K"]
        return {"bytes": 3 * n + 4 * case["rows"], "flops": 4 * n}
    if op == "dispatch":
        row = case["H"] + (4 if case["fmt"] == "int8" else case["H"] // 32)
        return {"bytes": case["T"] * row * (1 + case["k"]) + 4 * case["T"] * case["k"], "flops": 0}
    rows, N, K = case["T"] * case["k"], case["N"], case["K"]
    out = 2 * rows * (N // 2 if case["swiglu"] else N)
    return {"bytes": rows * (K + 4) + int(_experts_used(case) * N * (K + 4)) + out, "flops": 2 * rows * N * K}


# ---------------------------------------------------------------------------
# the definitions in 64 bits


def _np(t):
    return None if t is None else t.detach().double().cpu().numpy()


def _exact_scores(case, l):
    with np.errstate(over="ignore", invalid="ignore"):
        if case["score"] == "sigmoid":
            return np.where(l > -np.inf, 1.0 / (1.0 + np.exp(-l)), 0.0)
        m = l.max(1, keepdims=True)
        e = np.where(l > -np.inf, np.exp(l - np.where(m > -np.inf, m, 0.0)), 0.0)
        z = e.sum(1, keepdims=True)
        return e / np.where(z > 0, z, 1.0)


def _exact_route(case, s):
    l = _np(s["logits"])
    T, E = l.shape
    sc = _exact_scores(case, l)
    plain_order = not case["bias"] and not (case["top2"] and case["groups"] > 1)
    v = l.copy() if plain_order else sc + (_np(s["bias"])[None] if case["bias"] else 0.0)
    v[l == -np.inf] = -np.inf
    G = case["groups"]
    if G > 1:
        p = np.sort(v.reshape(T, G, E // G), axis=2)[:, :, ::-1]
        val = p[:, :, 0].copy()
        if case["top2"] and E // G > 1:
            two = p[:, :, 1] > -np.inf
            val[two] += p[:, :, 1][two]
        rank = np.argsort(np.argsort(-val, axis=1, kind="stable"), axis=1, kind="stable")
        v = np.where(np.repeat(rank < case["kept"], E // G, axis=1), v, -np.inf)
    k = case["k"]
    idx = np.full((T, k), -1, np.int64)
    best = np.argsort(-v, axis=1, kind="stable")[:, :k]
    ok = np.take_along_axis(v, best, 1) > -np.inf
    idx[:, :best.shape[1]] = np.where(ok, best, -1)
    w = _exact_shares(case, idx, l, sc) * case["scale"]
    return [idx.astype(np.int32), w] + ([sc] if case["scores"] else [])


def _exact_shares(case, idx, l, sc):
    ok = idx >= 0
    w = np.where(ok, np.take_along_axis(sc, np.maximum(idx, 0), 1), 0.0)
    if case["renorm"]:
        z = w.sum(1, keepdims=True)
        w = w / np.where(z > 0, z, 1.0)
    return w


def _exact_route_bwd(case, s):
    l, idx, gw = _np(s["logits"]), s["idx"].long().cpu().numpy(), _np(s["gw"]) * case["scale"]
    T, E = l.shape
    sc = _exact_scores(case, l)
    ok, t = idx >= 0, np.arange(T)[:, None] + np.zeros_like(idx)
    ds = np.zeros((T, E)) if s["gs"] is None else _np(s["gs"]).copy()
    w = _exact_shares(case, idx, l, sc)
    gw = np.where(ok, gw, 0.0)
    d = gw
    if case["renorm"]:
        z = np.where(ok, np.take_along_axis(sc, np.maximum(idx, 0), 1), 0.0).sum(1, keepdims=True)
        d = np.where(ok, (gw - (gw * w).sum(1, keepdims=True)) / np.where(z > 0, z, 1.0), 0.0)
    np.add.at(ds, (t[ok], idx[ok]), d[ok])
    if case["score"] == "sigmoid":
        return ds * sc * (1.0 - sc)
    return sc * (ds - (ds * sc).sum(1, keepdims=True))


def _exact_norm(case, s):
    h = _np(s["x"])
    out = []
    if case["residual"] != "none":
        h = h + _np(s["residual"])
        out.append(h)
        # the stream's value is what its type holds: that is what is normalised
        h = _np(torch.from_numpy(h).to(s["residual"].dtype))
    y = h / np.sqrt((h * h).mean(1, keepdims=True) + EPS) * _np(s["weight"])
    if case["y"]:
        out.append(y)
    if case["quant"] == "int8":
        a = np.abs(y).max(1)
        scale = np.where(a > 0, a / 127.0, 1.0)
        out += [np.clip(np.rint(y / scale[:, None]), -127, 127).astype(np.int8), scale]
    elif case["quant"] != "none":
        a = np.abs(y.reshape(y.shape[0], -1, 128)).max(2)
        scale = np.where(a > 0, a / 448.0, 1.0)
        if case["quant"] == "fp8_pow2":
            scale = np.where(a > 0, np.exp2(np.ceil(np.log2(scale))), 1.0)
        out += [y / np.repeat(scale, 128, axis=1), scale]
    return out


def _exact_norm_bwd(case, s):
    h, gy, w = _np(s["hidden"]), _np(s["gy"]), _np(s["weight"])
    r = 1.0 / np.sqrt((h * h).mean(1, keepdims=True) + EPS)
    g = gy * w
    gx = g * r - h * r ** 3 * (g * h).mean(1, keepdims=True)
    if s["gh"] is not None:
        gx = gx + _np(s["gh"])
    return [gx, (gy * h * r).sum(0)]


def _exact_quantize(case, s):
    x = _np(s["x"])
    a = np.abs(x).max(1)
    scale = np.where(a > 0, a / 127.0, 1.0)
    return [np.clip(np.rint(x / scale[:, None]), -127, 127).astype(np.int8), scale]


def _exact_dispatch(case, s):
    dst, k = s["dst"].cpu().numpy(), case["k"]
    codes, scales = s["codes"], _np(s["scales"])
    codes = codes.cpu().numpy() if case["fmt"] == "int8" else _np(codes)
    recv = np.zeros((s["recv"].shape[0], codes.shape[1]), codes.dtype)
    rs = np.zeros((recv.shape[0],) + scales.shape[1:])
    for j in range(k):
        recv[dst[j::k]] = codes
        rs[dst[j::k]] = scales
    return [recv, rs]


def _exact_gemm(case, s):
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    row = 0
    for e, n in enumerate(s["counts"]):
        lo = e * case["cap"] if case["layout"] == "ll" else row
        row += n
        if n == 0:
            continue
        x = s["x"][lo:lo + n].double() * s["xs"][lo:lo + n].double()[:, None]
        w = s["w"][e].double() * s["ws"][e].double()[:, None]
        h = x @ w.t().contiguous()
        if case["swiglu"]:
            h = h.view(n, -1, 2)
            h = h[..., 0] / (1.0 + torch.exp(-h[..., 0])) * h[..., 1]
        out[lo:lo + n] = h
    return out


_EXACT = dict(route=_exact_route, route_bwd=_exact_route_bwd, norm=_exact_norm, norm_bwd=_exact_norm_bwd,
              quantize=_exact_quantize, dispatch=_exact_dispatch, gemm=_exact_gemm)


def exact(case, seed):
    global own
    was, own = own, False   # the inputs alone: nothing of the library is made
    try:
        return _EXACT[case["op"]](case, prepare(case, seed))
    finally:
        own = was
