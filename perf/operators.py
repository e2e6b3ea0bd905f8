"""Cases that measure the operators around the low-precision Linear: RMSNorm with the residual's
addition and an 8-bit output (forward and backward), MXFP4 quantisation and products, and the global
gradient norm with clipping.

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
EMAX = {"e4m3": 8, "e5m2": 15, "e2m1": 2}
FP4_VALUES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
EPS = 1e-5

# The gradients of one decoder layer: q, o, k, v, gate, up, down projections and two norms.
LAYER = (4096 * 4096, 4096 * 4096, 4096 * 1024, 4096 * 1024, 4096 * 14336, 4096 * 14336,
         14336 * 4096, 4096, 4096)


def listed():
    return [
        # one token of a decode step: its norm, in the block-scaled form that the next product reads
        {"name": "norm_token_mx", "op": "norm", "rows": 1, "cols": 4096, "x": "bf16", "h": "bf16",
         "quant": "mx", "fmt": "e4m3"},
        # the norm in front of a 4096-hidden Linear in training, delayed per-tensor scaling
        {"name": "norm_train", "op": "norm", "rows": 16384, "cols": 4096, "x": "bf16", "h": "bf16",
         "quant": "tensor", "fmt": "e4m3"},
        # an odd hidden size and batch, fp32 residual stream, per-token scales
        {"name": "norm_ragged_row", "op": "norm", "rows": 1531, "cols": 1023, "x": "bf16",
         "h": "f32", "quant": "row", "fmt": "e4m3"},
        # backward of norm_train: dX in BF16 and as the E5M2 operand of the layer below
        {"name": "norm_bwd_train", "op": "norm_bwd", "rows": 16384, "cols": 4096, "x": "bf16",
         "h": "bf16", "q": True, "fmt": "e5m2"},
        # backward of a small odd-sized fp32 norm
        {"name": "norm_bwd_small", "op": "norm_bwd", "rows": 300, "cols": 1030, "x": "f32",
         "h": "f32", "q": False, "fmt": "e5m2"},
        # many small gradients (norms, biases, adapters): latency counts
        {"name": "clip_small", "op": "clip", "tensors": 24, "most": 5000, "layers": 0,
         "grad": "bf16", "out": "bf16", "max_norm": 1.0},
        # the gradients of two decoder layers, clipped into the fp32 main gradients
        {"name": "clip_layers", "op": "clip", "tensors": 0, "most": 1, "layers": 2,
         "grad": "bf16", "out": "f32", "max_norm": 1.0},
        # weights through MXFP4 and back (quantisation-aware training, 16-bit fallback of a layer)
        {"name": "fp4_roundtrip", "op": "fp4_cast", "rows": 14336, "cols": 4096, "x": "bf16"},
        # one token through a gate/up projection: FP8 activations, FP4 weights
        {"name": "fp4_token", "op": "fp4_linear", "M": 1, "N": 14336, "K": 4096, "fa": "e4m3"},
        # a few sequences decoding together, FP4 on both sides, an odd count
        {"name": "fp4_decode_13", "op": "fp4_linear", "M": 13, "N": 4096, "K": 14336,
         "fa": "e2m1"},
        # a prompt through a gate/up projection
        {"name": "fp4_prompt", "op": "fp4_linear", "M": 8192, "N": 14336, "K": 4096,
         "fa": "e2m1"},
        # forward and backward of a 4096-hidden Linear in MXFP4
        {"name": "fp4_train", "op": "fp4_train", "M": 16384, "N": 4096, "K": 4096},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_bwd", "clip", "fp4_cast", "fp4_linear", "fp4_linear",
                     "fp4_train"])
    if op in ("norm", "norm_bwd"):
        cols = _log(rng, 64, 14336)
        rows = min(_log(rng, 1, 16384), (1 << 26) // cols)
        types = rng.choice([("bf16", "bf16"), ("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
        case = {"op": op, "rows": rows, "cols": cols, "x": types[0], "h": types[1]}
        if op == "norm_bwd":
            return dict(case, q=rng.random() < 0.5, fmt=rng.choice(["e5m2", "e4m3"]))
        case["quant"] = rng.choice(["none", "tensor", "row", "mx"])
        case["fmt"] = "e4m3"
        if case["quant"] == "mx":
            case["cols"] = max(64, cols // 32 * 32)
        elif rng.random() < 0.5:
            case["cols"] = max(64, cols // 8 * 8)
        return case
    if op == "clip":
        return {"op": op, "tensors": rng.randint(1, 50), "most": _log(rng, 10, 4000000),
                "layers": 0, "grad": rng.choice(["bf16", "f32"]), "out": rng.choice(["bf16", "f32"]),
                "max_norm": rng.choice([0.5, 1.0, 1e9])}
    if op == "fp4_cast":
        cols = 32 * _log(rng, 2, 448)
        return {"op": op, "rows": min(_log(rng, 1, 16384), (1 << 25) // cols), "cols": cols,
                "x": rng.choice(["bf16", "f32"])}
    if op == "fp4_linear":
        return {"op": op, "M": _log(rng, 1, 8192), "N": 8 * _log(rng, 8, 1792),
                "K": 32 * _log(rng, 4, 448 if rng.random() < 0.5 else 128),
                "fa": rng.choice(["e2m1", "e4m3"])}
    return {"op": op, "M": 32 * _log(rng, 4, 256), "N": 32 * _log(rng, 4, 128),
            "K": 32 * _log(rng, 4, 128)}


# ------------------------------------------------------------------ inputs


class State:
    pass


def _randn(g, shape, std, dtype):
    return torch.randn(shape, generator=g, device=DEV, dtype=F32).mul_(std).to(dtype)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    s = State()
    s.case, op = case, case["op"]
    if op == "norm":
        R, C, xt, ht = case["rows"], case["cols"], DTYPES[case["x"]], DTYPES[case["h"]]
        s.x, s.res = _randn(g, (R, C), 0.5, xt), _randn(g, (R, C), 2.0, ht)
        s.gamma = (1.0 + _randn(g, (C,), 0.1, F32)).to(xt)
        s.h, s.rstd = torch.empty_like(s.res), torch.empty(R, device=DEV)
        s.y = torch.empty(R, C, dtype=xt, device=DEV)
        s.q = torch.empty(R, C, dtype=U8, device=DEV)
        # a delayed scale as the history of such tensors gives it
        s.scale = torch.full((1,), 64.0, device=DEV)
        s.amax, s.sat = torch.zeros(1, device=DEV), torch.zeros(1, dtype=torch.int64, device=DEV)
        s.row_scale, s.row_amax = torch.empty(R, device=DEV), torch.empty(R, device=DEV)
        s.mx_scales = torch.empty(R, max(1, C // 32), dtype=U8, device=DEV)
    elif op == "norm_bwd":
        R, C, xt, ht = case["rows"], case["cols"], DTYPES[case["x"]], DTYPES[case["h"]]
        s.dy, s.h = _randn(g, (R, C), 1e-3, xt), _randn(g, (R, C), 2.0, ht)
        s.dres = _randn(g, (R, C), 1e-3, ht)
        s.gamma = (1.0 + _randn(g, (C,), 0.1, F32)).to(xt)
        # what the forward kept
        s.rstd = torch.cat([(c.double().square().mean(1) + EPS).rsqrt().float()
                            for c in s.h.split(2048)])
        s.dx, s.dgamma = torch.empty_like(s.h), torch.empty(C, device=DEV)
        s.q = torch.empty(R, C, dtype=U8, device=DEV)
        s.scale = torch.full((1,), 16.0 * F8_MAX[case["fmt"]], device=DEV)
        s.amax, s.sat = torch.zeros(1, device=DEV), torch.zeros(1, dtype=torch.int64, device=DEV)
        s.work = None
    elif op == "clip":
        sizes = _clip_sizes(case)
        gt, ot = DTYPES[case["grad"]], DTYPES[case["out"]]
        # one tensor in eight has much larger gradients than the others
        s.grads = [_randn(g, (n,), 3e-2 if i % 8 == 7 else 1e-3, gt) for i, n in enumerate(sizes)]
        s.out = [torch.empty(n, dtype=ot, device=DEV) for n in sizes]
        s.norm, s.coef = torch.empty(1, device=DEV), torch.empty(1, device=DEV)
        s.work = None
    elif op == "fp4_cast":
        s.x = _blocks(g, case["rows"], case["cols"], 1.0, DTYPES[case["x"]])
        s.q = torch.empty(case["rows"], case["cols"] // 2, dtype=U8, device=DEV)
        s.scales = torch.empty(case["rows"], case["cols"] // 32, dtype=U8, device=DEV)
        s.y = torch.empty(case["rows"], case["cols"], dtype=BF, device=DEV)
    elif op == "fp4_linear":
        M, N, K = case["M"], case["N"], case["K"]
        s.x = _blocks(g, M, K, 1.0, BF)
        # the layer's weights, stored in MXFP4
        s.wq = torch.randint(0, 256, (N, K // 2), generator=g, device=DEV, dtype=U8)
        s.ws = torch.randint(117, 121, (N, K // 32), generator=g, device=DEV, dtype=U8)
        s.xq = torch.empty(M, K if case["fa"] == "e4m3" else K // 2, dtype=U8, device=DEV)
        s.xs = torch.empty(M, K // 32, dtype=U8, device=DEV)
        s.y = torch.empty(M, N, dtype=BF, device=DEV)
    else:
        M, N, K = case["M"], case["N"], case["K"]
        s.x, s.w = _blocks(g, M, K, 1.0, BF), _blocks(g, K, N, 0.02, BF)
        s.dy = _blocks(g, M, N, 1e-3, BF)
        s.layer = None
    return s


def _clip_sizes(case):
    g = torch.Generator()
    g.manual_seed(1)
    ragged = (case["most"] ** torch.rand(case["tensors"], generator=g)).long().tolist()
    return list(LAYER) * case["layers"] + ragged


def _blocks(g, rows, cols, std, dtype):
    """Normal values whose columns have different magnitudes, as activations' channels do."""
    x = _randn(g, (rows, cols), std, F32)
    return x.mul_(torch.exp2(torch.randint(-2, 3, (1, cols), generator=g, device=DEV).float())).to(dtype)


# ------------------------------------------------------------------ plain forms


def _two_to(e):
    """2^e in fp32 for whole e in [-126, 127], from the bits: exp2 may be a rounding off."""
    return ((e.to(torch.int32) + 127).clamp(min=0) << 23).view(F32)


def _mx(y, fmt):
    """Blocks of 32 of each row: (elements as values, E8M0 codes)."""
    r, c = y.shape
    b = y.reshape(r, c // 32, 32)
    amax = b.abs().amax(-1)
    _, e = torch.frexp(amax)
    code = torch.where(amax == 0, torch.zeros_like(e), (e - 1 - EMAX[fmt] + 127).clamp(0, 254))
    v = b * _two_to(127 - code).unsqueeze(-1)
    if fmt == "e2m1":
        a = v.abs().clamp(max=6.0)
        step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0)).to(y.dtype)
        v = torch.copysign(torch.round(a / step) * step, v)
    else:
        v = v.clamp(-F8_MAX[fmt], F8_MAX[fmt]).to(F8[fmt])
    return v.reshape(r, c), code.to(U8)


def _mx_values(y, fmt):
    """What the block-scaled form of ``y`` stands for, in y's type."""
    v, code = _mx(y, fmt)
    x = _two_to(code.int() - 127).unsqueeze(-1)
    return (v.to(y.dtype).reshape(*code.shape, 32) * x).reshape(y.shape)


def _fp4_values(q, scales):
    """Values of packed 4-bit codes [rows, cols / 2] with E8M0 codes [rows, cols / 32]."""
    table = torch.tensor(FP4_VALUES + tuple(-v for v in FP4_VALUES), dtype=F32, device=q.device)
    v = torch.stack([table[(q & 15).long()], table[(q >> 4).long()]], -1)
    x = _two_to(scales.int() - 127).unsqueeze(-1)
    return (v.reshape(*scales.shape, 32) * x).reshape(q.shape[0], -1)


def _norm_plain(s):
    c = s.case
    s.h = (s.x.float() + s.res.float()).to(s.res.dtype)
    hf = s.h.float()
    rstd = torch.rsqrt(hf.square().mean(1) + EPS)
    y = hf * rstd.unsqueeze(1) * s.gamma.float()
    out = {"h": s.h, "rstd": rstd}
    top = F8_MAX["e4m3"]
    if c["quant"] == "none":
        out["y"] = y.to(s.x.dtype)
    elif c["quant"] == "tensor":
        out["q"] = (y * s.scale).clamp(-top, top).to(F8["e4m3"])
        out["amax"] = y.abs().amax().reshape(1)
    elif c["quant"] == "row":
        amax = y.abs().amax(1)
        scale = torch.where(amax > 0, top / amax, torch.ones_like(amax))
        out["q"] = (y * scale.unsqueeze(1)).clamp(-top, top).to(F8["e4m3"])
        out["scale"], out["amax"] = scale, amax
    else:
        out["q"], code = _mx(y, "e4m3")
        out["scales"] = code.view(torch.float8_e8m0fnu)
    return out


def _norm_bwd_plain(s):
    c = s.case
    hf, dy = s.h.float(), s.dy.float()
    xhat = hf * s.rstd.unsqueeze(1)
    g = dy * s.gamma.float()
    d = s.rstd.unsqueeze(1) * (g - xhat * (g * xhat).mean(1, keepdim=True)) + s.dres.float()
    out = {"dx": d.to(s.h.dtype), "dgamma": (dy * xhat).sum(0)}
    if c["q"]:
        top = F8_MAX[c["fmt"]]
        out["q"] = (d * s.scale).clamp(-top, top).to(F8[c["fmt"]])
        out["amax"] = d.abs().amax().reshape(1)
    return out


def _clip_plain(s):
    total = torch.stack([g.double().square().sum() for g in s.grads]).sum()
    norm = total.sqrt()
    coef = (s.case["max_norm"] / (norm + 1e-6)).clamp(max=1.0).float()
    out = [(g.float() * coef).to(o.dtype) for g, o in zip(s.grads, s.out)]
    return {"out": out, "norm": norm.float().reshape(1), "coef": coef.reshape(1)}


def _fp4_train_plain(s):
    x, w, dy = s.x.float(), s.w.float(), s.dy.float()
    y = _mx_values(x, "e2m1") @ _mx_values(w.t().contiguous(), "e2m1").t()
    dx = _mx_values(dy, "e2m1") @ _mx_values(w, "e2m1").t()
    dw = _mx_values(x.t().contiguous(), "e2m1") @ _mx_values(dy.t().contiguous(), "e2m1").t()
    return {"y": y.to(BF), "dx": dx.to(BF), "dw": dw.to(BF)}


# ------------------------------------------------------------------ the package's entry points


def _norm_own(s):
    import delayed_scaling_gemm_amd as dsg

    c = s.case
    out = {"h": s.h, "rstd": s.rstd}
    f8 = s.q.view(F8["e4m3"])
    if c["quant"] == "none":
        dsg.fp8ds_rmsnorm(s.x, s.gamma, EPS, residual=s.res, h=s.h, y=s.y, rstd=s.rstd)
        out["y"] = s.y
    elif c["quant"] == "tensor":
        s.amax.zero_()
        dsg.fp8ds_rmsnorm(s.x, s.gamma, EPS, residual=s.res, h=s.h, rstd=s.rstd, fmt=dsg.E4M3,
                          scale=s.scale, q=s.q, amax=s.amax)
        out["q"], out["amax"] = f8, s.amax
    elif c["quant"] == "row":
        dsg.fp8ds_rmsnorm_rowwise(s.x, s.gamma, EPS, dsg.E4M3, 0, s.q, s.row_scale,
                                  amax=s.row_amax, residual=s.res, h=s.h, rstd=s.rstd)
        out["q"], out["scale"], out["amax"] = f8, s.row_scale, s.row_amax
    else:
        dsg.fp8ds_rmsnorm_mx(s.x, s.gamma, EPS, dsg.E4M3, s.q, s.mx_scales, residual=s.res, h=s.h,
                             rstd=s.rstd)
        out["q"], out["scales"] = f8, s.mx_scales.view(torch.float8_e8m0fnu)
    return out


def _norm_bwd_own(s):
    import delayed_scaling_gemm_amd as dsg

    c = s.case
    if s.work is None:
        s.work = torch.empty(dsg.fp8ds_rmsnorm_bwd_workspace(c["rows"], c["cols"]), dtype=U8,
                             device=DEV)
    out = {"dx": s.dx, "dgamma": s.dgamma}
    if c["q"]:
        s.amax.zero_()
        fmt = dsg.E5M2 if c["fmt"] == "e5m2" else dsg.E4M3
        dsg.fp8ds_rmsnorm_bwd(s.dy, s.h, s.rstd, s.gamma, s.dx, s.dgamma, s.work, dres=s.dres,
                              fmt=fmt, scale=s.scale, q=s.q, amax=s.amax)
        out["q"], out["amax"] = s.q.view(F8[c["fmt"]]), s.amax
    else:
        dsg.fp8ds_rmsnorm_bwd(s.dy, s.h, s.rstd, s.gamma, s.dx, s.dgamma, s.work, dres=s.dres)
    return out


def _clip_own(s):
    import delayed_scaling_gemm_amd as dsg

    if s.work is None:
        s.work = torch.empty(dsg.fp8ds_grad_norm_workspace(), dtype=U8, device=DEV)
    dsg.fp8ds_grad_norm(s.grads, s.case["max_norm"], s.norm, s.coef, s.work)
    dsg.fp8ds_grad_clip(s.grads, s.coef, s.out)
    return {"out": s.out, "norm": s.norm, "coef": s.coef}


def _fp4_linear_own(s):
    import delayed_scaling_gemm_amd as dsg

    c = s.case
    M, N, K = c["M"], c["N"], c["K"]
    if c["fa"] == "e4m3":
        fa = dsg.E4M3
        dsg.fp8ds_cast_mx(s.x, fa, s.xq, s.xs)
    else:
        fa = dsg.E2M1
        dsg.fp8ds_cast_mxfp4(s.x, s.xq, s.xs)
    dsg.fp8ds_gemm_mxfp4(M, N, K, s.xq, fa, K, s.xs, K // 32, s.wq, K, s.ws, K // 32, s.y, N)
    return s.y


def _fp4_train_own(s):
    from delayed_scaling_gemm_amd.linear import MXFP4Linear

    if s.layer is None:
        s.layer = MXFP4Linear(device=DEV)
    out = s.layer.step(s.x, s.w, s.dy)
    return {"y": out["y"], "dx": out["dx"], "dw": out["dw"]}


def run(state):
    s, op = state, state.case["op"]
    if op == "norm":
        return _norm_own(s) if own else _norm_plain(s)
    if op == "norm_bwd":
        return _norm_bwd_own(s) if own else _norm_bwd_plain(s)
    if op == "clip":
        return _clip_own(s) if own else _clip_plain(s)
    if op == "fp4_linear":
        if own:
            return _fp4_linear_own(s)
        return (_mx_values(s.x.float(), s.case["fa"]) @ _fp4_values(s.wq, s.ws).t()).to(BF)
    if op == "fp4_train":
        return _fp4_train_own(s) if own else _fp4_train_plain(s)
    if own:
        import delayed_scaling_gemm_amd as dsg

        dsg.fp8ds_cast_mxfp4(s.x, s.q, s.scales)
        dsg.fp8ds_dequant_mxfp4(s.q, s.scales, s.y)
        return s.y
    return _mx_values(s.x.float(), "e2m1").to(BF)


def work(case):
    size = {"bf16": 2, "f32": 4}
    op = case["op"]
    if op == "norm":
        n = case["rows"] * case["cols"]
        out = size[case["x"]] if case["quant"] == "none" else 1
        return {"bytes": n * (size[case["x"]] + 2 * size[case["h"]] + out), "flops": 6 * n}
    if op == "norm_bwd":
        n = case["rows"] * case["cols"]
        return {"bytes": n * (size[case["x"]] + 3 * size[case["h"]] + int(case["q"])),
                "flops": 12 * n}
    if op == "clip":
        n = sum(_clip_sizes(case))
        return {"bytes": n * (size[case["grad"]] + size[case["out"]]), "flops": 3 * n}
    if op == "fp4_cast":
        n = case["rows"] * case["cols"]
        return {"bytes": n * (size[case["x"]] + 2), "flops": 4 * n}
    M, N, K = case["M"], case["N"], case["K"]
    if op == "fp4_linear":
        return {"bytes": 2 * M * K + N * K * 17 / 32 + 2 * M * N, "flops": 2 * M * N * K}
    return {"bytes": 4 * (M * K + K * N) + 2 * M * N * 2, "flops": 6 * M * N * K}


# ------------------------------------------------------------------ the definitions in 64 bits


def _pow2(e):
    return ((e.long() + 1023) << 52).view(F64)


def _block_exponent(y, fmt):
    """The exponent of each block's scale, and y divided by it."""
    b = y.unflatten(1, (-1, 32))
    a = b.abs().amax(-1)
    e = torch.floor(torch.log2(torch.where(a > 0, a, torch.ones_like(a)))).to(torch.int32)
    e = e - (_pow2(e) > a).int() + (_pow2(e + 1) <= a).int()  # log2 may round across an integer
    e = torch.where(a > 0, (e - EMAX[fmt]).clamp(-127, 127), torch.full_like(e, -127))
    return e, b / _pow2(e).unsqueeze(-1)


def _exact_mx(y, fmt):
    """What the block-scaled form of y (64 bits) stands for: nearest element of the format, ties to
    the even code."""
    e, b = _block_exponent(y, fmt)
    if fmt == "e2m1":
        grid = torch.tensor(FP4_VALUES, dtype=F64, device=y.device)
        mid = (grid[1:] + grid[:-1]) / 2
        a = b.abs()
        k = torch.bucketize(a, mid, right=False)  # borders belong to the lower element ...
        tie = (k < 7) & (a == mid[k.clamp(max=6)])
        v = grid[torch.where(tie & (k % 2 == 1), k + 1, k)]  # ... unless its code is odd
        v = torch.where(b < 0, -v, v)
    else:  # the conversion of values that fp32 holds exactly
        v = b.clamp(-F8_MAX[fmt], F8_MAX[fmt]).float().to(F8[fmt]).double()
    return (v * _pow2(e).unsqueeze(-1)).flatten(1)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        h = (s.x.double() + s.res.double()).float().to(s.res.dtype)
        r = 1.0 / torch.sqrt((h.double() ** 2).sum(1) / case["cols"] + EPS)
        y = h.double() * r[:, None] * s.gamma.double()
        top = F8_MAX["e4m3"]
        out = {"h": h, "rstd": r}
        # 8-bit outputs as the values before their rounding: both sides' distance is then the
        # format's own, and not the few values that lie next to a border between two codes
        if case["quant"] == "none":
            out["y"] = y
        elif case["quant"] == "tensor":
            out["q"] = (y * float(s.scale)).clamp(-top, top)
            out["amax"] = y.abs().max().reshape(1)
        elif case["quant"] == "row":
            a = y.abs().max(1).values
            out["q"], out["scale"], out["amax"] = y * (top / a)[:, None], top / a, a
        else:
            e, b = _block_exponent(y, "e4m3")
            out["q"], out["scales"] = b.flatten(1).clamp(-top, top), _pow2(e)
        return out
    if op == "norm_bwd":
        r, n = s.rstd.double()[:, None], case["cols"]
        xhat = s.h.double() * r
        dxhat = s.dy.double() * s.gamma.double()
        d = r / n * (n * dxhat - xhat * (dxhat * xhat).sum(1, keepdim=True)) + s.dres.double()
        out = {"dx": d, "dgamma": (s.dy.double() * xhat).sum(0)}
        if case["q"]:
            out["amax"] = d.abs().max().reshape(1)
            # E5M2's own rounding is over the distance that tells anything; dx is the same values
            out["q"] = (d * float(s.scale)).clamp(-448, 448) if case["fmt"] == "e4m3" else None
        return out
    if op == "clip":
        norm = math.sqrt(sum(float((g.double() ** 2).sum()) for g in s.grads))
        coef = min(1.0, case["max_norm"] / (norm + 1e-6))
        one = {"norm": norm, "coef": coef}
        out = {k: torch.full((1,), v, dtype=F64, device=DEV) for k, v in one.items()}
        out["out"] = [g.double() * coef for g in s.grads]
        return out
    if op == "fp4_cast":
        return torch.cat([_exact_mx(c.double(), "e2m1") for c in s.x.split(4096)])
    if op == "fp4_linear":
        sign = torch.tensor([1.0, -1.0], dtype=F64, device=DEV)
        grid = torch.tensor(FP4_VALUES, dtype=F64, device=DEV)
        w = torch.empty(case["N"], case["K"], dtype=F64, device=DEV)
        for half in (0, 1):
            n = (s.wq.int() >> (4 * half)) & 15
            w[:, half::2] = grid[(n & 7).long()] * sign[(n >> 3).long()]
        w *= _pow2(s.ws.int() - 127).repeat_interleave(32, 1)
        return _exact_mx(s.x.double(), case["fa"]) @ w.t()
    x, w, dy = s.x.double(), s.w.double(), s.dy.double()

    def q(a):
        return _exact_mx(a, "e2m1")

    xt, wt, dyt = (q(a.t().contiguous()) for a in (x, w, dy))
    return {"y": q(x) @ wt.t(), "dx": q(dy) @ q(w).t(), "dw": xt @ dyt.t()}
