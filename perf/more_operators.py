"""Cases that measure the operators of the gated feed-forward block: its products with the activation
(forward and backward), the norms before and after it with gate and residual scale (forward and
backward), and Muon's orthogonalised update with the weights' step.

``run`` computes each operator in its plain form (elementary torch operations in fp32, one rounding
at the end) or, with ``own`` set, through the package's entry points.  ``exact`` gives the same
outputs from the definitions in 64 bits.
"""

import math

import torch

own = False

DEV = "cuda"
BF, F32, F64, U8 = torch.bfloat16, torch.float32, torch.float64, torch.uint8
DTYPES = {"bf16": BF, "f32": F32}
F8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
F8_MAX = {"e4m3": 448.0, "e5m2": 57344.0}
EPS, POST_EPS = 1e-5, 1e-6
ALPHA = 0.25                        # the residual scale
NS = (3.4445, -4.7750, 2.0315)      # Newton-Schulz coefficients, five steps
MU, NS_EPS = 0.95, 1e-7
LR, DECAY = 2e-3, 0.1


def listed():
    return [
        # one token of a decode step through gate and up, calibrated scales: latency and weights
        {"name": "ffn_token", "op": "ffn", "M": 1, "F": 14336, "K": 4096, "act": "silu", "out": "q"},
        # a few odd-sized sequences, a width that is no multiple of anything, 16-bit output
        {"name": "ffn_ragged", "op": "ffn", "M": 77, "F": 1001, "K": 1040, "act": "gelu",
         "out": "y"},
        # gate and up of a 4096-hidden layer in training, pre-activations kept
        {"name": "ffn_train", "op": "ffn", "M": 8192, "F": 14336, "K": 4096, "act": "silu",
         "out": "train"},
        # its backward pass: the down projection's dX through the activation, as the E5M2 operand
        {"name": "ffn_bwd_train", "op": "ffn_bwd", "M": 8192, "F": 14336, "H": 4096,
         "act": "silu", "out": "q"},
        # backward of a small block of odd size, 16-bit gradients
        {"name": "ffn_bwd_small", "op": "ffn_bwd", "M": 300, "F": 1037, "H": 528, "act": "gelu",
         "out": "d"},
        # one token of a decode step between two blocks, the next product's operand in MX blocks
        {"name": "sandwich_token_mx", "op": "sandwich", "rows": 1, "cols": 4096, "x": "bf16",
         "h": "bf16", "gate": True, "row_gate": False, "quant": "mx"},
        # between two blocks of a 4096-hidden model in training, delayed per-tensor scaling
        {"name": "sandwich_train", "op": "sandwich", "rows": 16384, "cols": 4096, "x": "bf16",
         "h": "bf16", "gate": True, "row_gate": False, "quant": "tensor"},
        # the backward pass of that, the branch's gradient as the E5M2 operand of the block below
        {"name": "sandwich_bwd_train", "op": "sandwich_bwd", "rows": 16384, "cols": 4096,
         "x": "bf16", "h": "bf16", "gate": True, "row_gate": False, "q": True},
        # a small backward pass, odd sizes, fp32 stream, a gate per token beside the channels'
        {"name": "sandwich_bwd_small", "op": "sandwich_bwd", "rows": 300, "cols": 1030, "x": "bf16",
         "h": "f32", "gate": True, "row_gate": True, "q": False},
        # Muon on an adapter-sized matrix, rows longer than columns: latency
        {"name": "muon_small", "op": "muon", "rows": 333, "cols": 130, "g": "bf16"},
        # Muon on one up projection
        {"name": "muon_up", "op": "muon", "rows": 4096, "cols": 14336, "g": "bf16"},
        # the step of that projection's master weights and its FP8 copies for the next forward
        {"name": "muon_apply_up", "op": "apply", "rows": 4096, "cols": 14336},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["ffn", "ffn", "ffn", "ffn_bwd", "ffn_bwd", "sandwich", "sandwich",
                     "sandwich_bwd", "muon", "muon", "apply"])
    if op in ("ffn", "ffn_bwd"):
        M, F = _log(rng, 1, 8192), _log(rng, 16, 14336)
        K = _log(rng, 32, 4096)
        if rng.random() < 0.7:
            F, K = max(16, F // 16 * 16), max(32, K // 16 * 16)
        act = rng.choice(["silu", "silu", "gelu"])
        if op == "ffn":
            return {"op": op, "M": M, "F": F, "K": K, "act": act,
                    "out": rng.choice(["q", "y", "train", "train"])}
        return {"op": op, "M": M, "F": F, "H": K, "act": act, "out": rng.choice(["q", "d"])}
    if op in ("sandwich", "sandwich_bwd"):
        cols = _log(rng, 64, 14336)
        rows = min(_log(rng, 1, 16384), (1 << 26) // cols)
        if rng.random() < 0.5:
            cols = cols // 8 * 8
        types = rng.choice([("bf16", "bf16"), ("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
        case = {"op": op, "rows": rows, "cols": cols, "x": types[0], "h": types[1],
                "gate": rng.random() < 0.7, "row_gate": rng.random() < 0.4}
        if op == "sandwich_bwd":
            return dict(case, q=rng.random() < 0.5)
        case["quant"] = rng.choice(["none", "tensor", "row", "mx"])
        if case["quant"] == "mx":
            case["cols"] = max(64, cols // 32 * 32)
        return case
    small, large = _log(rng, 16, 4096), _log(rng, 16, 14336)
    small, large = min(small, large), max(small, large)
    rows, cols = (small, large) if rng.random() < 0.6 else (large, small)
    if op == "muon":
        return {"op": op, "rows": rows, "cols": cols, "g": rng.choice(["bf16", "f32"])}
    return {"op": op, "rows": rows, "cols": cols}


# ------------------------------------------------------------------ inputs


class State:
    pass


def _randn(g, shape, std, dtype):
    return torch.randn(shape, generator=g, device=DEV, dtype=F32).mul_(std).to(dtype)


def _codes(values, scale, fmt):
    """FP8 codes of values [rows, cols], rows starting at multiples of 16 bytes."""
    rows, cols = values.shape
    store = torch.zeros(rows, (cols + 15) // 16 * 16, dtype=U8, device=DEV)
    top = F8_MAX[fmt]
    store[:, :cols] = values.mul(scale).clamp_(-top, top).to(F8[fmt]).view(U8)
    return store[:, :cols]


def _one(v):
    return torch.full((1,), v, device=DEV)


def _gradient(g, shape, std):
    """Gradients: near-normal, one value in a hundred ten times as large."""
    x = _randn(g, shape, std, F32)
    return torch.where(torch.rand(shape, generator=g, device=DEV) < 0.01, 10.0 * x, x)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    s = State()
    s.case, op = case, case["op"]
    if op == "ffn":
        M, F, K = case["M"], case["F"], case["K"]
        std, sw = 1.28 / math.sqrt(K), 64.0 * math.sqrt(K)
        s.sx, s.sw = _one(64.0), _one(sw)
        s.x = _codes(_randn(g, (M, K), 1.0, F32), 64.0, "e4m3")
        # weights stacked, gate above up, K-contiguous: the transposed copy that the cast writes
        s.w = _codes(_randn(g, (2 * F, K), std, F32), sw, "e4m3")
        s.scale, s.amax = _one(8.0), torch.zeros(1, device=DEV)
        s.gu = torch.empty(M, 2 * F, dtype=BF, device=DEV) if case["out"] == "train" else None
        s.y = torch.empty(M, F, dtype=BF, device=DEV) if case["out"] == "y" else None
        s.q = torch.empty(M, F, dtype=U8, device=DEV) if case["out"] != "y" else None
    elif op == "ffn_bwd":
        M, F, H = case["M"], case["F"], case["H"]
        s.sdy, s.sw = _one(16384.0), _one(4096.0)
        s.dy = _codes(_gradient(g, (M, H), 1e-3), 16384.0, "e5m2")
        s.w = _codes(_randn(g, (F, H), 0.02, F32), 4096.0, "e4m3")  # the down projection [in, out]
        s.gu = _randn(g, (M, 2 * F), 1.28, BF)
        s.scale, s.amax = _one(65536.0), torch.zeros(1, device=DEV)
        s.dgu = torch.empty(M, 2 * F, dtype=BF, device=DEV) if case["out"] == "d" else None
        s.q = torch.empty(M, 2 * F, dtype=U8, device=DEV) if case["out"] == "q" else None
    elif op in ("sandwich", "sandwich_bwd"):
        R, C, xt, ht = case["rows"], case["cols"], DTYPES[case["x"]], DTYPES[case["h"]]
        s.x = _randn(g, (R, C), 0.5, xt)
        s.post_gamma = (1.0 + _randn(g, (C,), 0.1, F32)).to(xt)
        s.gamma = (1.0 + _randn(g, (C,), 0.1, F32)).to(xt)
        s.gate = 0.5 + _randn(g, (C,), 0.2, F32) if case["gate"] else None
        s.row_gate = torch.rand(R, generator=g, device=DEV) if case["row_gate"] else None
        s.amax, s.work = torch.zeros(1, device=DEV), None
        if op == "sandwich":
            s.res = _randn(g, (R, C), 2.0, ht)
            s.h = torch.empty_like(s.res)
            s.post_rstd, s.rstd = torch.empty(R, device=DEV), torch.empty(R, device=DEV)
            s.y = torch.empty(R, C, dtype=xt, device=DEV)
            s.q = torch.empty(R, C, dtype=U8, device=DEV)
            s.scale = _one(64.0)
            s.row_scale, s.row_amax = torch.empty(R, device=DEV), torch.empty(R, device=DEV)
            s.mx_scales = torch.empty(R, max(1, C // 32), dtype=U8, device=DEV)
        else:
            s.h = _randn(g, (R, C), 2.0, ht)
            s.dy, s.dres = _randn(g, (R, C), 1e-3, xt), _randn(g, (R, C), 1e-3, ht)
            # what the forward kept
            s.post_rstd, s.rstd = (
                torch.cat([(c.double().square().mean(1) + e).rsqrt().float() for c in t.split(2048)])
                for t, e in ((s.x, POST_EPS), (s.h, EPS)))
            s.dh, s.dx = torch.empty_like(s.h), torch.empty_like(s.x)
            s.dgamma, s.dpost_gamma, s.dgate = (torch.empty(C, device=DEV) for _ in range(3))
            s.drow_gate = torch.empty(R, device=DEV)
            s.q = torch.empty(R, C, dtype=U8, device=DEV)
            s.scale = _one(16.0 * F8_MAX["e5m2"])
    elif op == "muon":
        R, C = case["rows"], case["cols"]
        # a gradient's spectrum: a few strong directions over many weak ones
        k = min(8, R, C)
        low = _randn(g, (R, k), 1.0, F32) @ _randn(g, (k, C), 1.0, F32)
        s.g = (1e-4 * (low + _randn(g, (R, C), 1.0, F32))).to(DTYPES[case["g"]])
        s.m = _randn(g, (R, C), 3e-4, F32)
        s.o = torch.empty(R, C, dtype=BF, device=DEV)
        s.work = None
    else:
        R, C = case["rows"], case["cols"]
        s.w = _randn(g, (R, C), 0.02, F32)
        s.o = _randn(g, (R, C), 1.0 / math.sqrt(max(R, C)), BF)
        s.scale, s.amax = _one(2048.0), torch.zeros(1, device=DEV)
        s.q = torch.empty(R, C, dtype=U8, device=DEV)
        s.q_t = torch.empty(C, R, dtype=U8, device=DEV)
    return s


def _adjust(case):
    """Muon's step relative to the learning rate: an update of AdamW's size."""
    return 0.2 * math.sqrt(max(case["rows"], case["cols"]))


# ------------------------------------------------------------------ plain forms


def _act(g, kind):
    """act(g) and act'(g)."""
    if kind == "silu":
        p = torch.sigmoid(g)
        return g * p, p * (1.0 + g * (1.0 - p))
    c = math.sqrt(2.0 / math.pi)
    t = torch.tanh(c * (g + 0.044715 * g * g * g))
    return 0.5 * g * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * g * (1.0 - t * t) * c * (1.0 + 0.134145 * g * g)


def _fp8(v, fmt):
    return v.clamp(-F8_MAX[fmt], F8_MAX[fmt]).to(F8[fmt])


def _ffn_plain(s):
    c = s.case
    F = c["F"]
    gu = s.x.view(F8["e4m3"]).float() @ s.w.view(F8["e4m3"]).float().t() * (1.0 / (s.sx * s.sw))
    a = _act(gu[:, :F], c["act"])[0] * gu[:, F:]
    if c["out"] == "y":
        return {"y": a.to(BF)}
    out = {"q": _fp8(a * s.scale, "e4m3")}
    if c["out"] == "train":
        out["gu"], out["amax"] = gu.to(BF), a.abs().amax().reshape(1)
    return out


def _ffn_bwd_plain(s):
    c = s.case
    F = c["F"]
    da = s.dy.view(F8["e5m2"]).float() @ s.w.view(F8["e4m3"]).float().t() * (1.0 / (s.sdy * s.sw))
    act, slope = _act(s.gu[:, :F].float(), c["act"])
    d = torch.cat([da * s.gu[:, F:].float() * slope, da * act], 1)
    if c["out"] == "d":
        return {"dgu": d.to(BF)}
    return {"q": _fp8(d * s.scale, "e5m2"), "amax": d.abs().amax().reshape(1)}


def _two_to(e):
    """2^e in fp32 for whole e in [-126, 127], from the bits: exp2 may be a rounding off."""
    return ((e.to(torch.int32) + 127).clamp(min=0) << 23).view(F32)


def _gates(s):
    k = ALPHA if s.gate is None else ALPHA * s.gate
    return k if s.row_gate is None else k * s.row_gate.unsqueeze(1)


def _sandwich_plain(s):
    c = s.case
    x = s.x.float()
    post_rstd = torch.rsqrt(x.square().mean(1) + POST_EPS)
    s.h = (s.res.float() + _gates(s) * (x * post_rstd.unsqueeze(1) * s.post_gamma.float())).to(s.res.dtype)
    hf = s.h.float()
    rstd = torch.rsqrt(hf.square().mean(1) + EPS)
    y = hf * rstd.unsqueeze(1) * s.gamma.float()
    out = {"h": s.h, "post_rstd": post_rstd, "rstd": rstd}
    if c["quant"] == "none":
        out["y"] = y.to(s.x.dtype)
    elif c["quant"] == "tensor":
        out["q"], out["amax"] = _fp8(y * s.scale, "e4m3"), y.abs().amax().reshape(1)
    elif c["quant"] == "row":
        amax = y.abs().amax(1)
        scale = torch.where(amax > 0, 448.0 / amax, torch.ones_like(amax))
        out["q"], out["scale"], out["amax"] = _fp8(y * scale.unsqueeze(1), "e4m3"), scale, amax
    else:
        b = y.reshape(y.shape[0], -1, 32)
        amax = b.abs().amax(-1)
        code = torch.where(amax == 0, 0, (torch.frexp(amax)[1] - 1 - 8 + 127).clamp(0, 254))
        out["q"] = _fp8(b * _two_to(127 - code).unsqueeze(-1), "e4m3").reshape(y.shape)
        out["scales"] = code.to(U8).view(torch.float8_e8m0fnu)
    return out


def _sandwich_bwd_plain(s):
    dy, r2, r1 = s.dy.float(), s.rstd.unsqueeze(1), s.post_rstd.unsqueeze(1)
    xh2, g2 = s.h.float() * r2, dy * s.gamma.float()
    dh = r2 * (g2 - xh2 * (g2 * xh2).mean(1, keepdim=True)) + s.dres.float()
    xh1, pg = s.x.float() * r1, s.post_gamma.float()
    g1 = _gates(s) * pg * dh
    dx = r1 * (g1 - xh1 * (g1 * xh1).mean(1, keepdim=True))
    t = dh * xh1 * ALPHA
    out = {"dh": dh.to(s.h.dtype), "dgamma": (dy * xh2).sum(0)}
    if s.row_gate is not None:
        out["drow_gate"] = (t * (pg if s.gate is None else pg * s.gate)).sum(1)
        t = t * s.row_gate.unsqueeze(1)
    S = t.sum(0)
    out["dpost_gamma"] = S if s.gate is None else S * s.gate
    if s.gate is not None:
        out["dgate"] = S * pg
    if s.case["q"]:
        out["q"], out["amax"] = _fp8(dx * s.scale, "e5m2"), dx.abs().amax().reshape(1)
    else:
        out["dx"] = dx.to(s.x.dtype)
    return out


def _muon_plain(s):
    g = s.g.float()
    s.m.mul_(MU).add_(g)
    x = g + MU * s.m
    tall = x.shape[0] > x.shape[1]
    if tall:
        x = x.t()
    x = x / (x.norm() + NS_EPS)
    a, b, c = NS
    for _ in range(5):
        A = x @ x.t()
        x = a * x + (b * A + c * (A @ A)) @ x
    return {"m": s.m, "o": (x.t() if tall else x).to(BF).contiguous()}


def _apply_plain(s):
    s.w.mul_(1.0 - LR * DECAY).sub_(s.o.float() * (LR * _adjust(s.case)))
    q = _fp8(s.w * s.scale, "e4m3")
    return {"w": s.w, "q": q, "q_t": q.t().contiguous(), "amax": s.w.abs().amax().reshape(1)}


# ------------------------------------------------------------------ the package's calls


def _ffn_own(s):
    import delayed_scaling_gemm_amd as dsg

    c = s.case
    act = dsg.ACT_SILU if c["act"] == "silu" else dsg.ACT_GELU
    if c["out"] == "y":
        dsg.fp8ds_gated_gemm(s.x, dsg.E4M3, s.sx, s.w, dsg.E4M3, s.sw, act, y=s.y)
        return {"y": s.y}
    if c["out"] == "q":
        dsg.fp8ds_gated_gemm(s.x, dsg.E4M3, s.sx, s.w, dsg.E4M3, s.sw, act, scale=s.scale, q=s.q)
        return {"q": s.q.view(F8["e4m3"])}
    s.amax.zero_()
    dsg.fp8ds_gated_gemm(s.x, dsg.E4M3, s.sx, s.w, dsg.E4M3, s.sw, act, gu=s.gu, scale=s.scale, q=s.q,
                         amax=s.amax)
    return {"q": s.q.view(F8["e4m3"]), "gu": s.gu, "amax": s.amax}


def _ffn_bwd_own(s):
    import delayed_scaling_gemm_amd as dsg

    c = s.case
    act = dsg.ACT_SILU if c["act"] == "silu" else dsg.ACT_GELU
    if c["out"] == "d":
        dsg.fp8ds_gated_gemm_bwd(s.dy, dsg.E5M2, s.sdy, s.w, dsg.E4M3, s.sw, act, s.gu, dgu=s.dgu)
        return {"dgu": s.dgu}
    s.amax.zero_()
    dsg.fp8ds_gated_gemm_bwd(s.dy, dsg.E5M2, s.sdy, s.w, dsg.E4M3, s.sw, act, s.gu, scale=s.scale,
                             q=s.q, amax=s.amax)
    return {"q": s.q.view(F8["e5m2"]), "amax": s.amax}


def _sandwich_own(s):
    import delayed_scaling_gemm_amd as dsg

    head = (s.x, s.post_gamma, POST_EPS, s.res, s.gamma, EPS, s.h)
    more = dict(alpha=ALPHA, gate=s.gate, row_gate=s.row_gate, post_rstd=s.post_rstd, rstd=s.rstd)
    out = {"h": s.h, "post_rstd": s.post_rstd, "rstd": s.rstd}
    quant = s.case["quant"]
    if quant == "none":
        dsg.fp8ds_rmsnorm_sandwich(*head, y=s.y, **more)
        out["y"] = s.y
    elif quant == "tensor":
        s.amax.zero_()
        dsg.fp8ds_rmsnorm_sandwich(*head, fmt=dsg.E4M3, scale=s.scale, q=s.q, amax=s.amax, **more)
        out["q"], out["amax"] = s.q.view(F8["e4m3"]), s.amax
    elif quant == "row":
        dsg.fp8ds_rmsnorm_sandwich_rowwise(*head, dsg.E4M3, 0, s.q, s.row_scale, amax=s.row_amax, **more)
        out["q"], out["scale"], out["amax"] = s.q.view(F8["e4m3"]), s.row_scale, s.row_amax
    else:
        dsg.fp8ds_rmsnorm_sandwich_mx(*head, dsg.E4M3, s.q, s.mx_scales, **more)
        out["q"], out["scales"] = s.q.view(F8["e4m3"]), s.mx_scales.view(torch.float8_e8m0fnu)
    return out


def _sandwich_bwd_own(s):
    import delayed_scaling_gemm_amd as dsg

    c = s.case
    if s.work is None:
        s.work = torch.empty(dsg.fp8ds_rmsnorm_sandwich_bwd_workspace(c["rows"], c["cols"]), dtype=U8,
                             device=DEV)
    out = {"dh": s.dh, "dgamma": s.dgamma, "dpost_gamma": s.dpost_gamma}
    more = dict(alpha=ALPHA, dres=s.dres)
    if s.gate is not None:
        more.update(gate=s.gate, dgate=s.dgate)
        out["dgate"] = s.dgate
    if s.row_gate is not None:
        more.update(row_gate=s.row_gate, drow_gate=s.drow_gate)
        out["drow_gate"] = s.drow_gate
    if c["q"]:
        s.amax.zero_()
        more.update(fmt=dsg.E5M2, scale=s.scale, q=s.q, amax=s.amax)
        out["q"], out["amax"] = s.q.view(F8["e5m2"]), s.amax
    else:
        more.update(dx=s.dx)
        out["dx"] = s.dx
    dsg.fp8ds_rmsnorm_sandwich_bwd(s.dy, s.h, s.rstd, s.gamma, s.x, s.post_rstd, s.post_gamma, s.dh,
                                   s.dgamma, s.dpost_gamma, s.work, **more)
    return out


def _muon_own(s):
    import delayed_scaling_gemm_amd as dsg

    if s.work is None:
        s.work = torch.empty(dsg.fp8ds_muon_workspace(*s.g.shape), dtype=U8, device=DEV)
    dsg.fp8ds_muon_direction(s.g, s.o, s.work, momentum=s.m, mu=MU, nesterov=True, steps=5)
    return {"m": s.m, "o": s.o}


def _apply_own(s):
    import delayed_scaling_gemm_amd as dsg

    s.amax.zero_()
    dsg.fp8ds_muon_apply(s.w, s.o, LR, weight_decay=DECAY, adjust=_adjust(s.case), fmt=dsg.E4M3,
                         scale=s.scale, q=s.q, q_t=s.q_t, amax=s.amax)
    return {"w": s.w, "q": s.q.view(F8["e4m3"]), "q_t": s.q_t.view(F8["e4m3"]), "amax": s.amax}


_RUN = {"ffn": (_ffn_plain, _ffn_own), "ffn_bwd": (_ffn_bwd_plain, _ffn_bwd_own),
        "sandwich": (_sandwich_plain, _sandwich_own),
        "sandwich_bwd": (_sandwich_bwd_plain, _sandwich_bwd_own),
        "muon": (_muon_plain, _muon_own), "apply": (_apply_plain, _apply_own)}


def run(state):
    return _RUN[state.case["op"]][1 if own else 0](state)


def work(case):
    size = {"bf16": 2, "f32": 4}
    op = case["op"]
    if op == "ffn":
        M, F, K = case["M"], case["F"], case["K"]
        out = {"q": 1, "y": 2, "train": 5}[case["out"]]
        return {"bytes": M * K + 2 * F * K + out * M * F, "flops": 4 * M * F * K}
    if op == "ffn_bwd":
        M, F, H = case["M"], case["F"], case["H"]
        return {"bytes": M * H + F * H + (6 if case["out"] == "q" else 8) * M * F,
                "flops": 2 * M * F * H}
    n = case["rows"] * case["cols"]
    if op == "sandwich":
        out = size[case["x"]] if case["quant"] == "none" else 1
        return {"bytes": n * (size[case["x"]] + 2 * size[case["h"]] + out), "flops": 12 * n}
    if op == "sandwich_bwd":
        out = 1 if case["q"] else size[case["x"]]
        return {"bytes": n * (2 * size[case["x"]] + 3 * size[case["h"]] + out), "flops": 25 * n}
    if op == "muon":
        m, k = min(case["rows"], case["cols"]), max(case["rows"], case["cols"])
        # X X^T and A A are symmetric: half of each
        return {"bytes": n * (size[case["g"]] + 8 + 2),
                "flops": 5 * (m * m * k + m * m * m + 2 * m * m * k)}
    return {"bytes": n * (4 + 2 + 4 + 2), "flops": 4 * n}


# ------------------------------------------------------------------ the definitions in 64 bits


def _exact_act(g, kind):
    """act and its derivative from exponentials alone."""
    if kind == "silu":
        e = torch.exp(-g)
        return g / (1.0 + e), (1.0 + e + g * e) / (1.0 + e) ** 2
    z = 2.0 * math.sqrt(2.0 / math.pi) * (g + 0.044715 * g ** 3)
    dz = 2.0 * math.sqrt(2.0 / math.pi) * (1.0 + 3 * 0.044715 * g ** 2)
    e = torch.exp(-z)                       # (1 + tanh(z / 2)) / 2 = 1 / (1 + e^-z)
    return g / (1.0 + e), 1.0 / (1.0 + e) + g * e * dz / (1.0 + e) ** 2


def _exact_ffn(s, c):
    F = c["F"]
    x, w = (t.view(F8["e4m3"]).double() for t in (s.x, s.w))
    d = 1.0 / (float(s.sx) * float(s.sw))
    g, u = x @ w[:F].t() * d, x @ w[F:].t() * d
    a = _exact_act(g, c["act"])[0] * u
    if c["out"] == "y":
        return {"y": a}
    # 8-bit outputs as the values before their rounding: both sides' distance is then the format's
    # own, and not the few values that lie next to a border between two codes
    out = {"q": (a * float(s.scale)).clamp(-448, 448)}
    if c["out"] == "train":
        out["gu"], out["amax"] = torch.cat([g, u], 1), a.abs().max().reshape(1)
    return out


def _exact_ffn_bwd(s, c):
    F = c["F"]
    da = s.dy.view(F8["e5m2"]).double() @ s.w.view(F8["e4m3"]).double().t()
    da /= float(s.sdy) * float(s.sw)
    act, slope = _exact_act(s.gu[:, :F].double(), c["act"])
    d = torch.cat([slope * s.gu[:, F:].double() * da, act * da], 1)
    if c["out"] == "d":
        return {"dgu": d}
    # (E5M2's own rounding is over the distance that tells anything)
    return {"q": None, "amax": d.abs().max().reshape(1)}


def _exact_sandwich(s, c):
    n = c["cols"]
    x = s.x.double()
    r1 = 1.0 / torch.sqrt((x ** 2).sum(1) / n + POST_EPS)
    branch = x * r1[:, None] * s.post_gamma.double() * ALPHA
    if s.gate is not None:
        branch = branch * s.gate.double()
    if s.row_gate is not None:
        branch = branch * s.row_gate.double()[:, None]
    h = (s.res.double() + branch).float().to(s.res.dtype)
    r2 = 1.0 / torch.sqrt((h.double() ** 2).sum(1) / n + EPS)
    y = h.double() * r2[:, None] * s.gamma.double()
    out = {"h": h, "post_rstd": r1, "rstd": r2}
    if c["quant"] == "none":
        out["y"] = y
    elif c["quant"] == "tensor":
        out["q"], out["amax"] = (y * float(s.scale)).clamp(-448, 448), y.abs().max().reshape(1)
    elif c["quant"] == "row":
        a = y.abs().max(1).values
        out["q"], out["scale"], out["amax"] = y * (448 / a)[:, None], 448 / a, a
    else:
        b = y.unflatten(1, (-1, 32))
        a = b.abs().amax(-1)
        e = torch.floor(torch.log2(a)).long()
        p = ((e + 1023) << 52).view(F64)
        e = e - (p > a).long() + (2 * p <= a).long()  # log2 may round across an integer
        p = ((e - 8 + 1023) << 52).view(F64)
        out["q"], out["scales"] = (b / p[..., None]).flatten(1).clamp(-448, 448), p
    return out


def _exact_sandwich_bwd(s, c):
    n = c["cols"]
    r1, r2 = s.post_rstd.double()[:, None], s.rstd.double()[:, None]
    pg, dy = s.post_gamma.double(), s.dy.double()
    gate = 1.0 if s.gate is None else s.gate.double()
    t = 1.0 if s.row_gate is None else s.row_gate.double()[:, None]

    def through(d, xhat, r):  # the norm's backward pass, d the gradient of xhat
        return r / n * (n * d - xhat * (d * xhat).sum(1, keepdim=True))

    xh2, xh1 = s.h.double() * r2, s.x.double() * r1
    dh = through(dy * s.gamma.double(), xh2, r2) + s.dres.double()
    dp = ALPHA * t * gate * dh
    dx = through(dp * pg, xh1, r1)
    out = {"dh": dh, "dgamma": (dy * xh2).sum(0), "dpost_gamma": (dp * xh1).sum(0)}
    if s.gate is not None:
        out["dgate"] = (ALPHA * t * dh * pg * xh1).sum(0)
    if s.row_gate is not None:
        out["drow_gate"] = (ALPHA * gate * dh * pg * xh1).sum(1)
    if c["q"]:
        out["q"], out["amax"] = None, dx.abs().max().reshape(1)
    else:
        out["dx"] = dx
    return out


def _exact_muon(s, c):
    g = s.g.double()
    m = MU * s.m.double() + g
    x = g + MU * m
    x = x / (torch.sqrt((x ** 2).sum()) + NS_EPS)
    wide = x.shape[0] <= x.shape[1]
    a, b, k = NS
    for _ in range(5):  # (X X^T) X = X (X^T X)
        A = x @ x.t() if wide else x.t() @ x
        P = b * A + k * (A @ A)
        x = a * x + (P @ x if wide else x @ P)
    return {"m": m, "o": x}


def _exact_apply(s, c):
    w = (1.0 - LR * DECAY) * s.w.double() - LR * _adjust(c) * s.o.double()
    q = (w * float(s.scale)).clamp(-448, 448)
    return {"w": w, "q": q, "q_t": q.t().contiguous(), "amax": w.abs().max().reshape(1)}


_EXACT = {"ffn": _exact_ffn, "ffn_bwd": _exact_ffn_bwd, "sandwich": _exact_sandwich,
          "sandwich_bwd": _exact_sandwich_bwd, "muon": _exact_muon, "apply": _exact_apply}


def exact(case, seed):
    return _EXACT[case["op"]](prepare(case, seed), case)
