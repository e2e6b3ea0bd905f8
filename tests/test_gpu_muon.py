"""Muon's direction and step (fp8ds_muon_direction, fp8ds_muon_apply) against the iteration in 64 bits.

Momentum is two fp32 roundings, in a fixed order: checked bit for bit.  The direction's products take
pairs of BF16: an operand is off by at most 2^-18 of itself (hi rounds to 2^-9, lo the rest to 2^-9 of
that), the missing lo lo term is 2^-18 of the product, the fp32 sums less.  A step makes
a X + b A X + c A A X, three terms with singular values of at most about 1.2, of these products: its
error is taken as 2^-17 (|a| + |b| + |c|) |X|_F (roundings of either sign add in squares).  A later
step takes an error along as it does X, by at most its polynomial's largest slope,
max |a + 3 b s^2 + 5 c s^4|, a at s = 0 for the usual coefficients.  The bound is the sum of the steps'
errors so taken along, over the result's norm, with the norms of the iteration in 64 bits.  (A bound
that took the result's norm to be sqrt(min(R, C)) was wrong for decaying spectra, whose weakest
directions are not near 1 after five steps.)  A BF16 output is the fp32 one rounded."""

import math

import pytest

torch = pytest.importorskip("torch")

import delayed_scaling_gemm_amd as dsg  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32, F64, U8 = torch.bfloat16, torch.float32, torch.float64, torch.uint8
USUAL = (3.4445, -4.7750, 2.0315)


def slope(a, b, c):
    s = torch.linspace(0, 1.2, 500, dtype=F64)
    return float((a + 3 * b * s ** 2 + 5 * c * s ** 4).abs().max())


def direction64(u, steps=5, coefs=None, eps=1e-7):
    """The direction, and how far (2-norm, relative) fp32 results may be from it."""
    x = u.double()
    x = x / (torch.sqrt((x * x).sum()) + eps)
    tall = x.shape[0] > x.shape[1]
    x = x.t() if tall else x
    err = 0.0
    for k in range(steps):
        a, b, c = coefs[k] if coefs else USUAL
        err = err * slope(a, b, c) + 2.0 ** -17 * (abs(a) + abs(b) + abs(c)) * float(x.norm())
        A = x @ x.t()
        x = a * x + (b * A + c * (A @ A)) @ x
    return (x.t() if tall else x).contiguous(), err / float(x.norm())


def work(R, C):
    # what it holds does not matter: all bytes of a NaN
    return torch.full((dsg.fp8ds_muon_workspace(R, C),), 0xFF, dtype=U8, device=DEV)


def matrix(R, C, kind, seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed + 31 * R + C)
    rn = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    if kind == "gauss":
        return rn(R, C)
    if kind == "strong":  # a few strong directions over many weak ones
        k = min(4, R, C)
        return rn(R, k) @ rn(k, C) + 0.05 * rn(R, C)
    if kind == "decay":
        m = min(R, C)
        s = torch.logspace(0, -3, m, device=DEV)
        x = rn(R, m) * s @ rn(m, C) if m > 1 else rn(R, C)
        return x
    return torch.where(torch.rand(R, C, generator=g, device=DEV) < 0.01, 100 * rn(R, C), rn(R, C))


def far(o, e):
    return float((o.double() - e).norm() / e.norm())


@pytest.mark.parametrize("kind", ["gauss", "strong", "decay", "tails"])
@pytest.mark.parametrize("R,C", [(1, 1), (1, 300), (300, 1), (5, 7), (64, 64), (65, 63), (17, 1000), (130, 333),
                                 (333, 130), (128, 2048), (700, 260), (512, 512), (256, 6000)])
def test_direction(R, C, kind):
    g = matrix(R, C, kind) * 1e-3
    e, bound = direction64(g)
    o = torch.empty(R, C, device=DEV)
    dsg.fp8ds_muon_direction(g, o, work(R, C))
    assert far(o, e) <= bound
    o16 = torch.empty(R, C, dtype=BF, device=DEV)
    dsg.fp8ds_muon_direction(g, o16, work(R, C))
    assert torch.equal(o16, o.to(BF))


# tiles of 128 and 256, with and without groups of steps
@pytest.mark.parametrize("R,C", [(1500, 1400), (3000, 3100), (1100, 9000), (9000, 1100), (2100, 7000)])
def test_direction_large(R, C):
    g = matrix(R, C, "strong")
    o = torch.empty(R, C, device=DEV)
    dsg.fp8ds_muon_direction(g, o, work(R, C))
    e, bound = direction64(g)
    assert far(o, e) <= bound


@pytest.mark.parametrize("steps", [1, 2, 3, 4, 6, 7, 16])
@pytest.mark.parametrize("R,C", [(70, 64), (64, 300)])
def test_steps_and_coefficients(R, C, steps):
    g = matrix(R, C, "gauss", steps)
    coefs = [(1.5 + 0.5 / (k + 1), -0.5 - 1.0 / (k + 1), 0.5 / (k + 1)) for k in range(steps)]
    for cs in (None, coefs):
        o = torch.empty(R, C, device=DEV)
        dsg.fp8ds_muon_direction(g, o, work(R, C), steps=steps, coefs=cs)
        e, bound = direction64(g, steps, cs)
        assert far(o, e) <= bound


@pytest.mark.parametrize("gt", [BF, F32])
@pytest.mark.parametrize("nesterov", [True, False])
def test_momentum(gt, nesterov):
    R, C, mu = 45, 77, 0.9
    m = torch.zeros(R, C, device=DEV)
    ref = torch.zeros(R, C, device=DEV)
    coef = torch.full((1,), 0.37, device=DEV)
    ws, o = work(R, C), torch.empty(R, C, device=DEV)
    for step in range(3):
        g = matrix(R, C, "gauss", step).to(gt)
        dsg.fp8ds_muon_direction(g, o, ws, momentum=m, mu=mu, nesterov=nesterov, grad_scale=0.125,
                                 grad_coef=coef)
        gs = g.float() * (torch.full((1,), 0.125, device=DEV) * coef)
        ref = ref * torch.tensor(mu, device=DEV) + gs
        assert torch.equal(m, ref)
        u = gs + torch.tensor(mu, device=DEV) * ref if nesterov else ref
        e, bound = direction64(u)
        assert far(o, e) <= bound


@pytest.mark.parametrize("R,C", [(40, 96), (33, 50), (300, 77)])
def test_strided_rows(R, C):
    """Parts of stacked matrices; what lies beside o stays."""
    for gt, pad in ((BF, 4), (F32, 3), (BF, C)):
        g = matrix(R, C, "gauss").to(gt)
        store = torch.full((R, C + pad), 1e30, device=DEV, dtype=gt)
        store[:, pad:] = g
        m, m2 = torch.ones(R, C, device=DEV), torch.ones(R, C, device=DEV)
        o, p = torch.empty(R, C, device=DEV, dtype=BF), torch.full((R, C + pad), 9.0, device=DEV, dtype=BF)
        dsg.fp8ds_muon_direction(g, o, work(R, C), momentum=m)
        dsg.fp8ds_muon_direction(store[:, pad:], p[:, :C], work(R, C), momentum=m2)
        assert torch.equal(m, m2) and torch.equal(p[:, :C], o) and (p[:, C:] == 9).all()


def test_scale_free_and_extreme_magnitudes():
    R, C = 50, 90
    g, ws = matrix(R, C, "gauss"), work(R, C)
    o, p = (torch.empty(R, C, device=DEV) for _ in range(2))
    dsg.fp8ds_muon_direction(g, o, ws, eps=1e-30)
    for s in (2.0 ** -60, 2.0 ** 60):  # squares beyond fp32 either way
        dsg.fp8ds_muon_direction(g * s, p, ws, eps=1e-30)
        assert far(p, o.double()) <= 1e-6
    dsg.fp8ds_muon_direction(torch.zeros_like(g), o, ws)
    assert (o == 0).all()


def test_skip_nan_and_repeat():
    R, C = 40, 200
    g, ws = matrix(R, C, "gauss"), work(R, C)
    m, o = torch.ones(R, C, device=DEV), torch.full((R, C), 7.0, device=DEV)
    for bad in (float("nan"), float("inf")):
        dsg.fp8ds_muon_direction(g, o, ws, momentum=m, grad_amax=torch.full((1,), bad, device=DEV))
        assert (m == 1).all() and (o == 7).all()
    dsg.fp8ds_muon_direction(g, o, ws, momentum=m, grad_amax=torch.ones(1, device=DEV))
    m2, o2 = torch.ones(R, C, device=DEV), torch.empty(R, C, device=DEV)
    dsg.fp8ds_muon_direction(g, o2, work(R, C), momentum=m2)
    assert torch.equal(m, m2) and torch.equal(o, o2)
    g[3, 4] = float("nan")
    dsg.fp8ds_muon_direction(g, o, ws)
    assert torch.isnan(o).all()


@pytest.mark.parametrize("ot", [BF, F32])
@pytest.mark.parametrize("R,C", [(1, 1), (33, 100), (128, 256), (300, 130), (256, 512)])
def test_apply(R, C, ot):
    w, o = matrix(R, C, "gauss") * 0.02, (matrix(R, C, "gauss", 1) * 0.05).to(ot)
    lr, wd, adj = 0.02, 0.1, 0.2 * math.sqrt(max(R, C))
    lr32, wd32, adj32 = (float(torch.tensor(v, dtype=F32)) for v in (lr, wd, adj))
    decay, step = (torch.tensor(v, dtype=F32, device=DEV) for v in (1 - lr32 * wd32, lr32 * adj32))
    want = decay * w - step * o.float()
    a = w.clone()
    dsg.fp8ds_muon_apply(a, o, lr, weight_decay=wd, adjust=adj)
    assert torch.equal(a, want)
    scale, used = torch.full((1,), 3000.0, device=DEV), torch.zeros(1, device=DEV)
    for fmt in (dsg.E4M3, dsg.E5M2):
        q, q2 = (torch.empty(R, C, dtype=U8, device=DEV) for _ in range(2))
        qt, qt2 = (torch.empty(C, R, dtype=U8, device=DEV) for _ in range(2))
        am, am2 = (torch.zeros(1, device=DEV) for _ in range(2))
        sat, sat2 = (torch.zeros(1, dtype=torch.int64, device=DEV) for _ in range(2))
        dsg.fp8ds_cast(want, fmt, scale, q2, qt2, amax=am2, sat_count=sat2)
        a = w.clone()
        dsg.fp8ds_muon_apply(a, o, lr, weight_decay=wd, adjust=adj, fmt=fmt, scale=scale, q=q, q_t=qt,
                             scale_used=used, amax=am, sat_count=sat)
        assert torch.equal(a, want) and torch.equal(q, q2) and torch.equal(qt, qt2)
        assert torch.equal(am, am2) and torch.equal(sat, sat2) and torch.equal(used, scale)
        # combined into; without the transposed copy; a skipped step still casts
        am.fill_(1e9)
        b, q3 = w.clone(), torch.empty_like(q)
        dsg.fp8ds_muon_apply(b, o, lr, weight_decay=wd, adjust=adj, fmt=fmt, scale=scale, q=q3, amax=am,
                             sat_count=sat)
        assert torch.equal(q3, q) and float(am) == 1e9 and int(sat) == 2 * int(sat2)
        c = w.clone()
        dsg.fp8ds_muon_apply(c, o, lr, weight_decay=wd, adjust=adj, fmt=fmt, scale=scale, q=q3, q_t=qt,
                             grad_amax=torch.full((1,), float("nan"), device=DEV))
        dsg.fp8ds_cast(w, fmt, scale, q2)
        assert torch.equal(c, w) and torch.equal(q3, q2) and torch.equal(qt, q2.t().contiguous())


def test_graph_streams_and_shared_workspace():
    R, C = 96, 320
    ws, o, m = work(R, C), torch.empty(R, C, dtype=BF, device=DEV), torch.zeros(R, C, device=DEV)
    gs = [matrix(R, C, "strong", i).to(BF) for i in range(3)]
    g = gs[0].clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dsg.fp8ds_muon_direction(g, o, ws, momentum=m)
    ref = torch.zeros(R, C, device=DEV)
    side = torch.cuda.Stream()
    for i in (0, 1, 2, 1):
        g.copy_(gs[i])
        graph.replay()
        torch.cuda.synchronize()
        e = torch.empty_like(o)
        torch.cuda.synchronize()
        dsg.fp8ds_muon_direction(gs[i], e, work(R, C), momentum=ref, stream=side)
        torch.cuda.synchronize()
        assert torch.equal(o, e) and torch.equal(m, ref)
