"""The norms around a gated residual addition (fp8ds_rmsnorm_sandwich, _rowwise, _mx, _bwd) against
their formulas in 64 bits.

Tolerances, in steps of u = 2^-24 (half a step of fp32).  r1 and r2 come from a sum of C squares added
in lanes of at most 32 and as a tree: off by at most (C / threads + 12) u < 48 u of the sum, half of
that in r, and 3 u of their own operations: 32 u.  p = (x r1) k t has k = gamma gate alpha: 6 further
roundings, so h is off by 40 u |p| + u (|res| + |p|) before its own rounding (2^-8 |h| in BF16, which
may fall the other way: then everything after it is computed from the stored h, and so is the
reference).  y = (h r2) gamma: 40 u |y|.
Backward: the stored h, r1, r2 are inputs.  A mean of C products is off by 60 u of the mean of the
magnitudes (48 for its sum, the rest its terms); dh by 64 u (|r2| (|g2| + |xh2| mean|g2 xh2|) + |dres|),
dx by what that makes of it through the second norm, 64 u each, which is bounded below by the same
expression with |dh| + its error; column sums over R rows in fp32, in at most R + 16 additions, by
(R + 80) u of the sum of magnitudes."""

import pytest

torch = pytest.importorskip("torch")

import delayed_scaling_gemm_amd as dsg  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32, F64, U8 = torch.bfloat16, torch.float32, torch.float64, torch.uint8
U = 2.0 ** -24
TYPES = {"bb": (BF, BF), "bf": (BF, F32), "ff": (F32, F32)}
EPS1, EPS2 = 1e-6, 1e-5


def inputs(R, C, types, gate, row_gate, seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed + 7 * R + C)
    xt, ht = TYPES[types]
    rn = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    d = dict(x=(0.5 * rn(R, C)).to(xt), res=(2 * rn(R, C)).to(ht), pg=(1 + 0.1 * rn(C)).to(xt),
             ga=1 + 0.1 * rn(C), gate=0.5 + 0.2 * rn(C) if gate else None,
             t=torch.rand(R, generator=g, device=DEV) if row_gate else None)
    if gate and C % 2 == 0:
        d["gate"] = d["gate"].to(BF)
    d["x"][:, ::9] *= 5  # channels of different size
    return d


def half(v, dtype):
    return (2.0 ** -8 if dtype == BF else U) * v.abs()


def k64(d, alpha):
    k = alpha * d["pg"].double()
    return k if d["gate"] is None else k * d["gate"].double()


def forward64(d, alpha):
    C = d["x"].shape[1]
    x = d["x"].double()
    r1 = 1 / torch.sqrt((x * x).sum(1) / C + EPS1)
    p = x * r1[:, None] * k64(d, alpha)
    if d["t"] is not None:
        p = p * d["t"].double()[:, None]
    return r1, p, d["res"].double() + p


def run_forward(d, alpha, **kw):
    R, C = d["x"].shape
    h = torch.empty_like(d["res"])
    r1, r2 = torch.empty(R, device=DEV), torch.empty(R, device=DEV)
    dsg.fp8ds_rmsnorm_sandwich(d["x"], d["pg"], EPS1, d["res"], d["ga"], EPS2, h, alpha=alpha,
                               gate=d["gate"], row_gate=d["t"], post_rstd=r1, rstd=r2, **kw)
    return h, r1, r2


SHAPES = [(1, 1), (3, 5), (1, 8), (5, 33), (64, 64), (7, 127), (19, 520), (33, 1023), (8, 2048), (3, 4100),
          (5, 8192), (2, 16384), (3, 20000), (2, 40001), (2, 33)]


@pytest.mark.parametrize("types", list(TYPES))
@pytest.mark.parametrize("R,C", SHAPES)
def test_forward(R, C, types):
    gate, row_gate = R % 2 == 1, C % 2 == 1 or R == 2
    d = inputs(R, C, types, gate, row_gate)
    alpha = 0.5 if R == 7 else -1.25
    y = torch.empty(R, C, device=DEV)
    h, r1, r2 = run_forward(d, alpha, y=y)
    e1, p, hx = forward64(d, alpha)
    assert ((r1.double() - e1).abs() <= 32 * U * e1).all()
    loose = 40 * U * p.abs() + U * (d["res"].double().abs() + p.abs())
    assert ((h.double() - hx).abs() <= loose + half(hx.abs() + loose, h.dtype)).all()
    hs = h.double()
    e2 = 1 / torch.sqrt((hs * hs).sum(1) / C + EPS2)
    assert ((r2.double() - e2).abs() <= 32 * U * e2).all()
    yx = hs * e2[:, None] * d["ga"].double()
    assert ((y.double() - yx).abs() <= 40 * U * yx.abs()).all()
    # in place, 16 bits, and every cast are functions of these, bit for bit
    inplace = dict(d, res=d["res"].clone())
    h2 = inplace["res"]
    y16 = torch.empty(R, C, dtype=BF, device=DEV)
    dsg.fp8ds_rmsnorm_sandwich(d["x"], d["pg"], EPS1, h2, d["ga"], EPS2, h2, alpha=alpha, gate=d["gate"],
                               row_gate=d["t"], y=y16)
    assert torch.equal(h2, h) and torch.equal(y16, y.to(BF))
    for fmt in (dsg.E4M3, dsg.E5M2):
        s, used = torch.full((1,), 300.0, device=DEV), torch.zeros(1, device=DEV)
        am, sat = torch.zeros(1, device=DEV), torch.zeros(1, dtype=torch.int64, device=DEV)
        q, q2 = (torch.empty(R, C, dtype=U8, device=DEV) for _ in range(2))
        h3, _, _ = run_forward(d, alpha, fmt=fmt, scale=s, q=q, scale_used=used, amax=am, sat_count=sat)
        am2, sat2 = torch.zeros(1, device=DEV), torch.zeros_like(sat)
        dsg.fp8ds_cast(y, fmt, s, q2, amax=am2, sat_count=sat2)
        assert torch.equal(h3, h) and torch.equal(q, q2) and torch.equal(am, am2)
        assert torch.equal(sat, sat2) and torch.equal(used, s)
        rs, ri, ra = (torch.empty(R, device=DEV) for _ in range(3))
        ps, pi, pa = (torch.empty(R, device=DEV) for _ in range(3))
        dsg.fp8ds_rmsnorm_sandwich_rowwise(d["x"], d["pg"], EPS1, d["res"], d["ga"], EPS2, h3, fmt, 1, q,
                                           rs, ri, ra, alpha=alpha, gate=d["gate"], row_gate=d["t"])
        dsg.fp8ds_cast_rowwise(y, fmt, 1, q2, ps, pi, pa)
        assert torch.equal(q, q2) and torch.equal(rs, ps) and torch.equal(ri, pi) and torch.equal(ra, pa)
    if C % 32 == 0:
        for fmt in (dsg.E4M3, dsg.E5M2, dsg.E2M1):
            n = C // 2 if fmt == dsg.E2M1 else C
            q, q2 = (torch.empty(R, n, dtype=U8, device=DEV) for _ in range(2))
            sc, sc2 = (torch.empty(R, C // 32, dtype=U8, device=DEV) for _ in range(2))
            pg = d["pg"]
            dsg.fp8ds_rmsnorm_sandwich_mx(d["x"], pg, EPS1, d["res"], d["ga"], EPS2, h3, fmt, q, sc,
                                          alpha=alpha, gate=d["gate"], row_gate=d["t"])
            if fmt == dsg.E2M1:
                dsg.fp8ds_cast_mxfp4(y, q2, sc2)
            else:
                dsg.fp8ds_cast_mx(y, fmt, q2, sc2)
            assert torch.equal(q, q2) and torch.equal(sc, sc2) and torch.equal(h3, h)


def backward64(dy, h, r2, d, r1, alpha, dres):
    """Gradients in 64 bits and their bounds."""
    C = h.shape[1]
    dy, h, r2, x, r1 = dy.double(), h.double(), r2.double()[:, None], d["x"].double(), r1.double()[:, None]
    t = 1.0 if d["t"] is None else d["t"].double()[:, None]
    ga, pg, k = d["ga"].double(), d["pg"].double(), k64(d, alpha)
    gate = 1.0 if d["gate"] is None else d["gate"].double()
    xh2, g2 = h * r2, dy * ga
    dh = r2 * (g2 - xh2 * (g2 * xh2).mean(1, keepdim=True))
    edh = 64 * U * r2.abs() * (g2.abs() + xh2.abs() * (g2 * xh2).abs().mean(1, keepdim=True))
    if dres is not None:
        dh, edh = dh + dres.double(), edh + 64 * U * dres.double().abs()
    xh1 = x * r1
    dp = k * dh                                     # before the token's factor
    m = (dp * xh1).mean(1, keepdim=True)
    em = ((k.abs() * (edh + 64 * U * dh.abs()) * xh1.abs()).mean(1, keepdim=True))
    dx = t * r1 * (dp - xh1 * m)
    mag = (t * r1 * (dp.abs() + xh1.abs() * (dp * xh1).abs().mean(1, keepdim=True))).abs()
    edx = 64 * U * mag + (t * r1 * (k.abs() * edh + xh1.abs() * em)).abs()
    n = h.shape[0] + 80
    S = alpha * t * dh * xh1
    eS = (abs(alpha) * t * edh * xh1.abs() + n * U * S.abs()).sum(0)
    out = {"dh": dh, "dx": dx, "dgamma": (dy * xh2).sum(0), "dpost_gamma": (gate * S).sum(0),
           "dgate": (pg * S).sum(0), "drow_gate": m[:, 0] * C}
    tol = {"dh": edh, "dx": edx, "dgamma": (n * U * (dy * xh2).abs()).sum(0) + 1e-37,
           "dpost_gamma": abs(gate) * eS * (1 + 4 * U) + 1e-37, "dgate": pg.abs() * eS * (1 + 4 * U) + 1e-37,
           "drow_gate": em[:, 0] * C + 64 * U * (dp * xh1).abs().sum(1)}
    return out, tol


def run_backward(d, h, r1, r2, dy, alpha, dres, **kw):
    R, C = h.shape
    o = {"dh": torch.empty_like(h), "dgamma": torch.empty(C, device=DEV),
         "dpost_gamma": torch.empty(C, device=DEV)}
    if d["gate"] is not None:
        o["dgate"] = torch.empty(C, device=DEV)
    if d["t"] is not None:
        o["drow_gate"] = torch.empty(R, device=DEV)
    ws = torch.full((dsg.fp8ds_rmsnorm_sandwich_bwd_workspace(R, C),), 0xFF, dtype=U8, device=DEV)
    dsg.fp8ds_rmsnorm_sandwich_bwd(dy, h, r2, d["ga"], d["x"], r1, d["pg"], o["dh"], o["dgamma"],
                                   o["dpost_gamma"], ws, alpha=alpha, gate=d["gate"], row_gate=d["t"],
                                   dgate=o.get("dgate"), drow_gate=o.get("drow_gate"), dres=dres, **kw)
    return o


@pytest.mark.parametrize("types", list(TYPES))
@pytest.mark.parametrize("R,C", SHAPES + [(1500, 72), (300, 1030)])
def test_backward(R, C, types):
    gate, row_gate = R % 2 == 1, C % 2 == 1 or R == 2
    d = inputs(R, C, types, gate, row_gate, seed=1)
    alpha = 0.75
    h, r1, r2 = run_forward(d, alpha)
    g = torch.Generator(device=DEV).manual_seed(R * C)
    dy = torch.randn(R, C, generator=g, device=DEV).to(d["x"].dtype)
    dres = torch.randn(R, C, generator=g, device=DEV).to(h.dtype) if R != 5 else None
    dx = torch.empty(R, C, device=DEV, dtype=d["x"].dtype)
    got = run_backward(d, h, r1, r2, dy, alpha, dres, dx=dx)
    got["dx"] = dx
    want, tol = backward64(dy, h, r2, d, r1, alpha, dres)
    for name, v in got.items():
        e = tol[name]
        assert ((v.double() - want[name]).abs() <= e + half(want[name].abs() + e, v.dtype)).all(), name
    # in place (dh over dres, dx over dy), with the cast, whose codes are those of the fp32 dx
    s, used = torch.full((1,), 50.0, device=DEV), torch.zeros(1, device=DEV)
    am, sat = torch.zeros(1, device=DEV), torch.zeros(1, dtype=torch.int64, device=DEV)
    q = torch.empty(R, C, dtype=U8, device=DEV)
    dy2 = dy.clone()
    again = run_backward(d, h, r1, r2, dy2, alpha, dres, dx=dy2, scale=s, q=q, scale_used=used, amax=am,
                         sat_count=sat)
    again["dx"] = dy2
    for name, v in got.items():
        assert torch.equal(v, again[name]), name
    if dres is not None:
        o, d2 = {k: torch.empty_like(v) for k, v in got.items()}, dres.clone()
        ws = torch.empty(dsg.fp8ds_rmsnorm_sandwich_bwd_workspace(R, C), dtype=U8, device=DEV)
        dsg.fp8ds_rmsnorm_sandwich_bwd(dy, h, r2, d["ga"], d["x"], r1, d["pg"], d2, o["dgamma"],
                                       o["dpost_gamma"], ws, alpha=alpha, gate=d["gate"],
                                       row_gate=d["t"], dres=d2)
        assert torch.equal(d2, got["dh"])
    if d["x"].dtype == F32:
        q2, am2, sat2 = torch.empty_like(q), torch.zeros_like(am), torch.zeros_like(sat)
        dsg.fp8ds_cast(dx, dsg.E5M2, s, q2, amax=am2, sat_count=sat2)
        assert torch.equal(q, q2) and torch.equal(am, am2) and torch.equal(sat, sat2)
    assert torch.equal(used, s)


def test_gradients_against_differences():
    """The whole operator's gradients against central differences of it in 64 bits."""
    R, C, alpha = 3, 24, 0.5
    d = inputs(R, C, "ff", True, True, seed=3)
    d["gate"] = d["gate"].float()
    g = torch.Generator(device=DEV).manual_seed(9)
    dy = torch.randn(R, C, generator=g, device=DEV)
    h, r1, r2 = run_forward(d, alpha)
    dx = torch.empty(R, C, device=DEV)
    got = run_backward(d, h, r1, r2, dy, alpha, None, dx=dx)

    def loss(v):
        r = 1 / torch.sqrt((v["x"] ** 2).mean(1, keepdim=True) + EPS1)
        hh = v["res"] + alpha * v["gate"] * v["t"][:, None] * v["pg"] * v["x"] * r
        s = 1 / torch.sqrt((hh ** 2).mean(1, keepdim=True) + EPS2)
        return float((dy.double() * hh * s * v["ga"]).sum())

    base = {k: v.double() for k, v in d.items()}
    names = {"x": dx, "res": got["dh"], "pg": got["dpost_gamma"], "ga": got["dgamma"],
             "gate": got["dgate"], "t": got["drow_gate"]}
    step = 1e-5
    for name, grad in names.items():
        for i in range(0, base[name].numel(), 5):
            up, down = ({k: v.clone() for k, v in base.items()} for _ in range(2))
            up[name].view(-1)[i] += step
            down[name].view(-1)[i] -= step
            num = (loss(up) - loss(down)) / (2 * step)
            # 2^-52 of a sum below 1e3 over the step: 2e-8; step^2 of third derivatives below 1e3:
            # 2e-8; fp32 sums of 72 terms below 30: 1e-4
            assert abs(num - float(grad.view(-1)[i])) <= 2e-4, (name, i)


def test_nan_rows_and_zero_rows():
    R, C = 9, 264
    d = inputs(R, C, "bb", True, False)
    d["x"][2, 5] = float("nan")
    d["x"][4] = 0
    d["res"][4] = 0
    d["x"][6, 0] = float("inf")
    q, sc = torch.empty(R, C, dtype=U8, device=DEV), torch.empty(R, device=DEV)
    y, h = torch.empty(R, C, device=DEV), torch.empty_like(d["res"])
    dsg.fp8ds_rmsnorm_sandwich_rowwise(d["x"], d["pg"], EPS1, d["res"], d["ga"], EPS2, h, dsg.E4M3, 0, q, sc,
                                       gate=d["gate"], y=y)
    assert torch.isnan(y[2]).all() and (y[4] == 0).all() and (q[4] == 0).all() and torch.isnan(y[6]).any()
    ok = [0, 1, 3, 5, 7, 8]
    clean = {k: (v[ok].clone() if v is not None and v.dim() == 2 else v) for k, v in d.items()}
    y2, h2 = torch.empty(len(ok), C, device=DEV), torch.empty_like(clean["res"])
    dsg.fp8ds_rmsnorm_sandwich(clean["x"], d["pg"], EPS1, clean["res"], d["ga"], EPS2, h2, gate=d["gate"],
                               y=y2)
    assert torch.equal(y[ok], y2) and torch.equal(h[ok], h2)


def test_strided_rows_streams_and_graph():
    R, C, alpha = 21, 100, 0.5
    d = inputs(R, C, "bb", True, True)
    y = torch.empty(R, C, device=DEV)
    h, r1, r2 = run_forward(d, alpha, y=y)
    dy, dres = torch.randn(R, C, device=DEV).to(BF), torch.randn(R, C, device=DEV).to(BF)
    want = run_backward(d, h, r1, r2, dy, alpha, dres)

    def wide(t, pad):
        s = torch.full((t.shape[0] + 1, t.shape[1] + pad), 3, dtype=t.dtype, device=DEV)
        s[:t.shape[0], :t.shape[1]] = t
        return s[:t.shape[0], :t.shape[1]]

    for pad in (1, 4, 28):
        e = dict(d, x=wide(d["x"], pad), res=wide(d["res"], pad))
        hv, yv = wide(torch.zeros_like(h), pad), wide(torch.zeros_like(y), pad)
        dsg.fp8ds_rmsnorm_sandwich(e["x"], e["pg"], EPS1, e["res"], e["ga"], EPS2, hv, alpha=alpha,
                                   gate=e["gate"], row_gate=e["t"], y=yv)
        assert torch.equal(hv, h) and torch.equal(yv, y)
        assert (hv._base[R] == 3).all() and (hv._base[:, C:] == 3).all()
        assert (yv._base[R] == 3).all() and (yv._base[:, C:] == 3).all()
        o = run_backward(e, hv, r1, r2, wide(dy, pad), alpha, wide(dres, pad))
        for k in want:
            assert torch.equal(o[k], want[k]), k
    # a graph of forward and backward on a side stream, replayed on new inputs between eager calls
    x = d["x"].clone()
    e = dict(d, x=x)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        gy = torch.empty(R, C, device=DEV)
        gh, g1, g2 = run_forward(e, alpha, y=gy)
        go = run_backward(e, gh, g1, g2, dy, alpha, dres)
    for i in range(3):
        x.copy_(torch.randn(R, C, device=DEV).to(BF))
        graph.replay()
        torch.cuda.synchronize()
        ey = torch.empty(R, C, device=DEV)
        eh, e1, e2 = run_forward(e, alpha, y=ey)
        eo = run_backward(e, eh, e1, e2, dy, alpha, dres)
        torch.cuda.synchronize()
        assert torch.equal(ey, gy) and torch.equal(eh, gh)
        assert all(torch.equal(eo[k], go[k]) for k in eo)


def test_no_rows():
    C = 40
    z = torch.empty(0, C, dtype=BF, device=DEV)
    v, r = torch.ones(C, device=DEV), torch.empty(0, device=DEV)
    used, s = torch.zeros(1, device=DEV), torch.full((1,), 2.0, device=DEV)
    dsg.fp8ds_rmsnorm_sandwich(z, v, EPS1, z, v, EPS2, z, scale=s, q=z.view(U8)[:, :C], scale_used=used)
    assert float(used) == 2.0
    dg, dp, dt = (torch.full((C,), 5.0, device=DEV) for _ in range(3))
    dsg.fp8ds_rmsnorm_sandwich_bwd(z, z, r, v, z, r, v, z, dg, dp, torch.empty(0, dtype=U8, device=DEV),
                                   gate=v, dgate=dt)
    assert (dg == 0).all() and (dp == 0).all() and (dt == 0).all()


def test_many_rows_go_round_the_grid():
    """More rows than a grid's workgroups take at a time: every one as alone."""
    R, C = 9000, 520
    d = inputs(R, C, "bb", True, True)
    y = torch.empty(R, C, device=DEV)
    h, r1, r2 = run_forward(d, 0.5, y=y)
    dy = torch.randn(R, C, device=DEV).to(BF)
    o = run_backward(d, h, r1, r2, dy, 0.5, None)
    for lo in (0, 4096, R - 37):
        part = {k: (v[lo:lo + 37] if v is not None and v.shape[0] == R else v) for k, v in d.items()}
        y2 = torch.empty(37, C, device=DEV)
        h2, _, _ = run_forward(part, 0.5, y=y2)
        assert torch.equal(h2, h[lo:lo + 37]) and torch.equal(y2, y[lo:lo + 37])
        o2 = run_backward(part, h2, r1[lo:lo + 37], r2[lo:lo + 37], dy[lo:lo + 37], 0.5, None)
        assert torch.equal(o2["dh"], o["dh"][lo:lo + 37])
        assert torch.equal(o2["drow_gate"], o["drow_gate"][lo:lo + 37])
    want, tol = backward64(dy, h, r2, d, r1, 0.5, None)
    for k in ("dgamma", "dpost_gamma", "dgate"):
        assert ((o[k].double() - want[k]).abs() <= tol[k]).all(), k


@pytest.mark.parametrize("types", list(TYPES))
@pytest.mark.parametrize("R,C", [(700, 33), (700, 777), (600, 2049), (300, 5003), (300, 9063)])
def test_ragged_rows_in_place_are_the_others(R, C, types):
    """Many ragged rows, every output that may lie over an input doing so: the same bits."""
    d = inputs(R, C, types, True, True, seed=5)
    h, r1, r2 = run_forward(d, 0.5)
    over = d["res"].clone()
    am, am2 = torch.zeros(1, device=DEV), torch.zeros(1, device=DEV)
    s = torch.full((1,), 20.0, device=DEV)
    q, q2 = (torch.empty(R, C, dtype=U8, device=DEV) for _ in range(2))
    run_forward(d, 0.5, fmt=dsg.E4M3, scale=s, q=q, amax=am)
    dsg.fp8ds_rmsnorm_sandwich(d["x"], d["pg"], EPS1, over, d["ga"], EPS2, over, alpha=0.5, gate=d["gate"],
                               row_gate=d["t"], fmt=dsg.E4M3, scale=s, q=q2, amax=am2)
    assert torch.equal(over, h) and torch.equal(q, q2) and torch.equal(am, am2)
    g = torch.Generator(device=DEV).manual_seed(C)
    dy = torch.randn(R, C, generator=g, device=DEV).to(d["x"].dtype)
    dres = torch.randn(R, C, generator=g, device=DEV).to(h.dtype)
    dx = torch.empty_like(dy)
    am, am2 = torch.zeros(1, device=DEV), torch.zeros(1, device=DEV)
    got = run_backward(d, h, r1, r2, dy, 0.5, dres, dx=dx, scale=s, q=q, amax=am)
    dy2, d2 = dy.clone(), dres.clone()
    o = {k: torch.empty_like(v) for k, v in got.items()}
    ws = torch.empty(dsg.fp8ds_rmsnorm_sandwich_bwd_workspace(R, C), dtype=U8, device=DEV)
    dsg.fp8ds_rmsnorm_sandwich_bwd(dy2, h, r2, d["ga"], d["x"], r1, d["pg"], d2, o["dgamma"],
                                   o["dpost_gamma"], ws, alpha=0.5, gate=d["gate"], row_gate=d["t"],
                                   dgate=o["dgate"], drow_gate=o["drow_gate"], dres=d2, dx=dy2, scale=s,
                                   q=q2, amax=am2)
    o["dh"] = d2
    for name, v in got.items():
        assert torch.equal(v, o[name]), name
    assert torch.equal(dx, dy2) and torch.equal(q, q2) and torch.equal(am, am2)
