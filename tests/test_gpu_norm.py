"""GPU parity of the RMSNorm calls against the fp64 oracle (oracle/norm.py).

Tolerances, derived from the kernels' sums with u = 2^-24 (half an fp32 step): a lane
adds at most 64 squares in order (long rows: cols / 1024), lanes are joined in 6 + 16
additions, so the sum of squares is off by at most (chain + 24) u relative, r by half
of that and 3 u for the division, root and reciprocal, y by 2 u more:
    T(cols) = (max(64, cols / 1024) / 2 + 20) u   relative, for r and y.
A code is right if it lies between the codes of y (1 - T) s and y (1 + T) s."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import delayed_scaling_gemm_amd as dsg  # noqa: E402
from oracle import bf16 as obf16  # noqa: E402
from oracle import fp8 as ofp8  # noqa: E402
from oracle import mx as omx  # noqa: E402
from oracle import mxfp4 as o4  # noqa: E402
from oracle import norm as onorm  # noqa: E402
from oracle import scaling as oscaling  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0**-24
EPS = 1e-5
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
PAIRS = [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")]


def tol(cols):
    return (max(64, cols / 1024) / 2 + 20) * U


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def make(rows, cols, xt, ht, seed, spread=True):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((rows, cols))
    res = 2.0 * rng.standard_normal((rows, cols))
    if spread:  # rows of very different magnitude
        m = 2.0 ** rng.integers(-12, 13, (rows, 1))
        x, res = x * m, res * m
    g = 1.0 + 0.2 * rng.standard_normal(cols)
    to = lambda a, t: torch.from_numpy(a).to(DEV).to(TYPES[t])  # noqa: E731
    return to(x, xt), to(res, ht), to(g, xt)


def check_y(got, y, cols, bf16_out):
    err = np.abs(got - y)
    bound = tol(cols) * np.abs(y) * (1 + 2.0**-8)
    if bf16_out:  # one rounding: half a step of 2^-7 at most
        bound = bound + np.abs(y) * 2.0**-8 + 2.0**-134
    assert (err <= bound).all(), (err - bound).max()


def between(codes, y, s, t, decode, encode):
    """Every decoded code lies between the roundings of y s (1 -+ t)."""
    s = np.asarray(s, np.float64)
    # two more fp32 roundings: the product with the scale, and the given s itself is exact
    lo = encode(np.asarray(y * s * (1 - t - 2 * U), np.float32))
    hi = encode(np.asarray(y * s * (1 + t + 2 * U), np.float32))
    d, a, b = decode(codes), decode(lo), decode(hi)
    assert ((d >= np.minimum(a, b)) & (d <= np.maximum(a, b))).all()


def fp8(fmt):
    return (lambda c: ofp8.decode(c, fmt)), (lambda v: ofp8.encode(v, fmt))


SHAPES = [(1, 1), (1, 4096), (3, 7), (5, 128), (17, 100), (33, 256), (9, 1000), (6, 1030),
          (4, 2048), (7, 4096), (3, 4100), (2, 8192), (600, 8192), (2, 14336), (2, 32768), (2, 40000),
          (1, 33001), (300, 64)]


@pytest.mark.parametrize("xt,ht", PAIRS)
@pytest.mark.parametrize("shape", SHAPES)
def test_y_h_rstd_and_tensor_scale(shape, xt, ht):
    rows, cols = shape
    x, res, g = make(rows, cols, xt, ht, rows * 7 + cols)
    for with_res in (True, False):
        h = torch.empty(rows, cols, dtype=TYPES[ht], device=DEV)
        y = torch.empty(rows, cols, dtype=TYPES[xt], device=DEV)
        r = torch.empty(rows, device=DEV)
        q = torch.empty(rows, cols, dtype=torch.uint8, device=DEV)
        sc = torch.tensor([37.0], device=DEV)
        used, am = torch.zeros(1, device=DEV), torch.zeros(1, device=DEV)
        sat = torch.zeros(1, dtype=torch.int64, device=DEV)
        fmt = dsg.E5M2 if (rows + cols) % 2 else dsg.E4M3
        dsg.fp8ds_rmsnorm(x, g, EPS, residual=res if with_res else None, h=h, y=y, rstd=r, fmt=fmt,
                          scale=sc, q=q, scale_used=used, amax=am, sat_count=sat)
        torch.cuda.synchronize()
        hr = onorm.residual_sum(f64(x), f64(res) if with_res else None, ht == "bf16")
        assert np.array_equal(f64(h), hr)
        rr, yr = onorm.forward(hr, f64(g), EPS)
        assert (np.abs(f64(r) - rr) <= tol(cols) * rr).all()
        check_y(f64(y), yr, cols, xt == "bf16")
        between(q.cpu().numpy(), yr, 37.0, tol(cols), *fp8(fmt))
        a = np.abs(yr).max()
        assert abs(float(am) - a) <= tol(cols) * a and float(used) == 37.0
        lim = ofp8.fmt_max(fmt)
        yl = np.abs(yr) * 37.0
        lo, hi = (yl > lim * (1 + tol(cols))).sum(), (yl > lim * (1 - tol(cols))).sum()
        assert lo <= int(sat) <= hi


@pytest.mark.parametrize("xt,ht", PAIRS)
@pytest.mark.parametrize("shape", [(1, 4096), (5, 100), (33, 256), (3, 1023), (9, 4096), (4, 8192),
                                   (2, 33001)])
@pytest.mark.parametrize("fmt", [dsg.E4M3, dsg.E5M2])
def test_rowwise(shape, xt, ht, fmt):
    rows, cols = shape
    x, res, g = make(rows, cols, xt, ht, rows + 3 * cols)
    if rows > 4:
        x[2] = 0
        res[2] = 0
    margin = rows % 3 - 1
    q = torch.empty(rows, cols, dtype=torch.uint8, device=DEV)
    s, si, am = (torch.empty(rows, device=DEV) for _ in range(3))
    dsg.fp8ds_rmsnorm_rowwise(x, g, EPS, fmt, margin, q, s, scale_inv=si, amax=am, residual=res)
    torch.cuda.synchronize()
    hr = onorm.residual_sum(f64(x), f64(res), ht == "bf16")
    _, yr = onorm.forward(hr, f64(g), EPS)
    a = np.abs(yr).max(axis=1)
    assert (np.abs(f64(am) - a) <= tol(cols) * a).all()
    ref = np.array([oscaling.scale_from_window(np.float32(v), fmt, margin)
                    for v in am.cpu().numpy()], np.float32)
    assert np.array_equal(s.cpu().numpy(), ref)
    assert np.array_equal(si.cpu().numpy(), np.float32(1.0) / ref)
    between(q.cpu().numpy(), yr, ref[:, None].astype(np.float64), tol(cols), *fp8(fmt))


@pytest.mark.parametrize("xt,ht", PAIRS)
@pytest.mark.parametrize("shape", [(1, 4096), (5, 32), (33, 96), (3, 992), (9, 4096), (4, 14336),
                                   (2, 32800)])
@pytest.mark.parametrize("fmt", [dsg.E4M3, dsg.E5M2, dsg.E2M1])
def test_mx(shape, xt, ht, fmt):
    rows, cols = shape
    x, res, g = make(rows, cols, xt, ht, rows + 5 * cols + fmt)
    g[:32] *= 2.0**-20  # a small block
    if cols > 64:
        g[32:64] = 0    # a zero block
    w = cols // 2 if fmt == dsg.E2M1 else cols
    q = torch.empty(rows, w, dtype=torch.uint8, device=DEV)
    s = torch.empty(rows, cols // 32, dtype=torch.uint8, device=DEV)
    h = torch.empty(rows, cols, dtype=TYPES[ht], device=DEV)
    dsg.fp8ds_rmsnorm_mx(x, g, EPS, fmt, q, s, residual=res, h=h)
    torch.cuda.synchronize()
    hr = onorm.residual_sum(f64(x), f64(res), ht == "bf16")
    assert np.array_equal(f64(h), hr)
    _, yr = onorm.forward(hr, f64(g), EPS)
    am = np.abs(yr.reshape(rows, -1, 32)).max(axis=2)
    emax = 2 if fmt == dsg.E2M1 else omx.EMAX_ELEM[fmt]

    def code(a):
        e = np.frexp(a)[1] - 1 - emax
        return np.where(a == 0, 0, np.clip(e, -127, 127) + 127)

    got = s.cpu().numpy().astype(np.int64)
    t = tol(cols)
    assert ((got >= code(am * (1 - t))) & (got <= code(am * (1 + t)))).all()
    inv = np.repeat(np.ldexp(1.0, 127 - got), 32, axis=1)
    qc = q.cpu().numpy()
    if fmt == dsg.E2M1:
        between(o4.unpack(qc), yr, inv, t, o4.decode, o4.encode)
    else:
        between(qc, yr, inv, t, *fp8(fmt))


def test_strided_rows_and_in_place():
    rows, cols = 37, 520
    x, res, g = make(rows, cols, "bf16", "bf16", 5)
    wide = torch.zeros(rows, 3 * cols + 8, dtype=torch.bfloat16, device=DEV)
    xs, rs, ys = wide[:, 8:8 + cols], wide[:, 8 + cols:8 + 2 * cols], wide[:, 8 + 2 * cols:]
    xs.copy_(x)
    rs.copy_(res)
    qw = torch.full((rows, cols + 24), 9, dtype=torch.uint8, device=DEV)
    one, y0 = torch.ones(1, device=DEV), torch.empty_like(x)
    q0, h0 = torch.empty(rows, cols, dtype=torch.uint8, device=DEV), torch.empty_like(x)
    dsg.fp8ds_rmsnorm(x, g, EPS, residual=res, h=h0, y=y0, scale=one, q=q0)
    dsg.fp8ds_rmsnorm(xs, g, EPS, residual=rs, h=rs, y=ys, scale=one, q=qw[:, 8:8 + cols])
    torch.cuda.synchronize()
    assert torch.equal(rs, h0) and torch.equal(ys, y0) and torch.equal(qw[:, 8:8 + cols], q0)
    assert (qw[:, :8] == 9).all() and (qw[:, 8 + cols:] == 9).all() and torch.equal(xs, x)
    # the same values at odd addresses: another layout of lanes, sums within the tolerance
    flat = torch.zeros(rows * cols + 1, dtype=torch.bfloat16, device=DEV)
    xo = flat[1:].view(rows, cols)
    xo.copy_(x)
    yo = torch.empty_like(x)
    dsg.fp8ds_rmsnorm(xo, g, EPS, residual=res, y=yo)
    torch.cuda.synchronize()
    check_y(f64(yo), onorm.forward(f64(h0), f64(g), EPS)[1], cols, True)


def test_long_rows_in_place():
    rows, cols = 2, 36000
    x, res, g = make(rows, cols, "bf16", "bf16", 6)
    h0, y0, y1 = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x)
    dsg.fp8ds_rmsnorm(x, g, EPS, residual=res, h=h0, y=y0)
    r2 = res.clone()
    dsg.fp8ds_rmsnorm(x, g, EPS, residual=r2, h=r2, y=y1)
    torch.cuda.synchronize()
    assert torch.equal(r2, h0) and torch.equal(y1, y0)


@pytest.mark.parametrize("cols", [96, 4096, 36000])
def test_non_finite_rows_stay_in_their_rows(cols):
    x, res, g = make(4, cols, "bf16", "bf16", 9)
    x[1, 5], x[2, 40] = float("nan"), float("inf")
    q = torch.empty(4, cols, dtype=torch.uint8, device=DEV)
    s = torch.empty(4, cols // 32, dtype=torch.uint8, device=DEV)
    rs, am = torch.empty(4, device=DEV), torch.zeros(1, device=DEV)
    dsg.fp8ds_rmsnorm_mx(x, g, EPS, dsg.E4M3, q, s, residual=res)
    torch.cuda.synchronize()
    sc = s.cpu().numpy()
    # NaN reaches every element through r; an infinite sum gives r = 0: Inf * 0 in one block
    assert (sc[1] == 255).all() and sc[2, 1] == 255 and (sc[[0, 3]] != 255).all()
    assert (q.cpu().numpy()[1] == 0x7F).all() and (np.delete(sc[2], 1) == 0).all()
    dsg.fp8ds_rmsnorm_rowwise(x, g, EPS, dsg.E4M3, 0, q, rs, residual=res)
    dsg.fp8ds_rmsnorm(x, g, EPS, residual=res, scale=torch.ones(1, device=DEV), q=q, amax=am)
    torch.cuda.synchronize()
    assert float(rs[1]) == 1.0 and float(rs[2]) == 1.0 and np.isnan(float(am))
    assert am.cpu().numpy().view(np.uint32)[0] == 0x7FC00000
    c = q.cpu().numpy()
    assert ((c[1] & 0x7F) == 0x7F).all() and ((c[[0, 3]] & 0x7F) != 0x7F).all()


def test_zero_rows_and_empty_inputs():
    g = torch.ones(64, device=DEV)
    x = torch.zeros(3, 64, device=DEV)
    y, r = torch.full_like(x, 5.0), torch.empty(3, device=DEV)
    dsg.fp8ds_rmsnorm(x, g, EPS, y=y, rstd=r)
    torch.cuda.synchronize()
    assert (y == 0).all() and torch.allclose(r, torch.full_like(r, EPS**-0.5))
    used = torch.zeros(1, device=DEV)
    e = torch.empty(0, 64, device=DEV)
    dsg.fp8ds_rmsnorm(e, g, EPS, y=torch.empty_like(e), scale=torch.full((1,), 3.0, device=DEV),
                      q=torch.empty(0, 64, dtype=torch.uint8, device=DEV), scale_used=used)
    dg = torch.full((64,), 7.0, device=DEV)
    dsg.fp8ds_rmsnorm_bwd(e, e, torch.empty(0, device=DEV), g, torch.empty_like(e), dg, None)
    torch.cuda.synchronize()
    assert float(used) == 3.0 and (dg == 0).all()


# ------------------------------------------------------------------ backward


def run_bwd(dy, h, r, g, dres=None, **kw):
    rows, cols = h.shape
    n = dsg.fp8ds_rmsnorm_bwd_workspace(rows, cols)
    work = torch.full((max(n, 1),), 0xFF, dtype=torch.uint8, device=DEV)  # NaN if read unwritten
    dx, dg = torch.empty_like(h), torch.empty(cols, device=DEV)
    dsg.fp8ds_rmsnorm_bwd(dy, h, r, g, dx, dg, work, dres=dres, **kw)
    torch.cuda.synchronize()
    return dx, dg


@pytest.mark.parametrize("xt,ht", PAIRS)
@pytest.mark.parametrize("shape", [(1, 1), (1, 4096), (3, 7), (300, 128), (17, 100), (33, 500),
                                   (1500, 1030), (9, 2048), (2100, 512), (40, 4096), (5, 8192),
                                   (3, 14336), (3, 17000), (2, 40000)])
def test_backward(shape, xt, ht):
    """dx off by at most 200 u of the absolute terms (a dot product of 64 + 24 links, and
    the products around it), dgamma by (rows a thread adds + 70) u of its absolute sum."""
    rows, cols = shape
    _, h, g = make(rows, cols, xt, ht, rows + 11 * cols, spread=False)
    dy, dres, _ = make(rows, cols, xt, ht, rows + 13 * cols)
    r = torch.from_numpy((1 / np.sqrt((f64(h)**2).mean(1) + EPS)).astype(np.float32)).to(DEV)
    for with_res in (True, False):
        am = torch.zeros(1, device=DEV)
        q = torch.empty(rows, cols, dtype=torch.uint8, device=DEV)
        sc = torch.tensor([0.25], device=DEV)
        fmt = dsg.E4M3 if rows % 2 else dsg.E5M2
        dx, dg = run_bwd(dy, h, r, g, dres if with_res else None, fmt=fmt, scale=sc, q=q, amax=am)
        ex, eg, terms = onorm.backward(f64(dy), f64(h), f64(r), f64(g),
                                       f64(dres) if with_res else None)
        slack = max(200, cols / 1024 + 150) * U * terms
        err = np.abs(f64(dx) - ex)
        assert (err <= slack + (np.abs(ex) + slack) * (2.0**-8 if ht == "bf16" else U)).all()
        a = np.abs(ex)
        assert abs(float(am) - a.max()) <= slack.max()
        lo, hi = ((ex - slack) * 0.25).astype(np.float32), ((ex + slack) * 0.25).astype(np.float32)
        d = ofp8.decode(q.cpu().numpy(), fmt)
        dlo, dhi = (ofp8.decode(ofp8.encode(v, fmt), fmt) for v in (lo, hi))
        assert ((d >= dlo) & (d <= dhi)).all()
        mag = (np.abs(f64(dy)) * np.abs(f64(h)) * f64(r)[:, None]).sum(0)
        assert (np.abs(f64(dg) - eg) <= (min(rows, rows / 1024 + 1024) + 70) * U * mag).all()


def test_backward_same_bits_again_and_aliases():
    _, h, g = make(700, 1024, "bf16", "bf16", 3, spread=False)
    dy, dres, _ = make(700, 1024, "bf16", "bf16", 4)
    r = torch.rand(700, device=DEV) + 0.5
    a, b = run_bwd(dy, h, r, g, dres), run_bwd(dy, h, r, g, dres)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    work = torch.empty(dsg.fp8ds_rmsnorm_bwd_workspace(700, 1024), dtype=torch.uint8, device=DEV)
    dg = torch.empty(1024, device=DEV)
    d2 = dres.clone()
    dsg.fp8ds_rmsnorm_bwd(dy, h, r, g, d2, dg, work, dres=d2)
    torch.cuda.synchronize()
    assert torch.equal(d2, a[0]) and torch.equal(dg, a[1])


def test_gradient_against_differences():
    """The backward kernel against differences of the forward kernel (fp32, a small shape):
    a central difference of step 2^-6 is off by its third-order term and by the loss's own
    rounding over the step."""
    rows, cols = 2, 40
    x, _, g = make(rows, cols, "f32", "f32", 21, spread=False)
    dy, _, _ = make(rows, cols, "f32", "f32", 22, spread=False)
    y, r = torch.empty_like(x), torch.empty(rows, device=DEV)

    def loss(xv):
        dsg.fp8ds_rmsnorm(xv, g, EPS, y=y, rstd=r)
        return float((y.double() * dy.double()).sum())

    loss(x)
    dx, _ = run_bwd(dy, x, r.clone(), g)
    step = 2.0**-6
    for i, j in ((0, 0), (0, 17), (1, 39), (1, 20)):
        e = torch.zeros_like(x)
        e[i, j] = step
        d = (loss(x + e) - loss(x - e)) / (2 * step)
        # third order: step^2 / 6 times a derivative of order 10; rounding: 80 values of
        # magnitude ~3 off by 40 u over 2 step
        assert abs(d - float(dx[i, j])) < 10 * step**2 / 6 + 80 * 3 * 40 * U / (2 * step)


def test_graph_replays_and_streams():
    x, res, g = make(64, 1024, "bf16", "bf16", 31)
    h, q = torch.empty_like(x), torch.empty(64, 1024, dtype=torch.uint8, device=DEV)
    sc, am = torch.ones(1, device=DEV), torch.zeros(1, device=DEV)
    r, dg, dx = torch.empty(64, device=DEV), torch.empty(1024, device=DEV), torch.empty_like(x)
    work = torch.empty(dsg.fp8ds_rmsnorm_bwd_workspace(64, 1024), dtype=torch.uint8, device=DEV)

    def both():
        dsg.fp8ds_rmsnorm(x, g, EPS, residual=res, h=h, rstd=r, scale=sc, q=q, amax=am)
        dsg.fp8ds_rmsnorm_bwd(x, h, r, g, dx, dg, work)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        both()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    for k in range(3):
        x.copy_(torch.randn(64, 1024, device=DEV))
        am.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (h, q, am, r, dx, dg)]
        am.zero_()
        both()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, (h, q, am, r, dx, dg))), k


@pytest.mark.parametrize("ht", ["bf16", "f32"])
@pytest.mark.parametrize("cols", [4096, 12288, 16400, 20481, 32768])
def test_many_rows_equal_few_at_a_time(cols, ht):
    """Workgroups that go on to further rows give what they give for the first."""
    rows, part = 600, 75
    x, res, g = make(rows, cols, "bf16", ht, cols)
    s = torch.full((1,), 8.0, device=DEV)

    def run(a, b):
        n = b - a
        h, y = torch.empty(n, cols, dtype=TYPES[ht], device=DEV), torch.empty(n, cols, device=DEV)
        q = torch.empty(n, cols, dtype=torch.uint8, device=DEV)
        r, am = torch.empty(n, device=DEV), torch.zeros(1, device=DEV)
        dsg.fp8ds_rmsnorm(x[a:b], g, EPS, res[a:b], h, y, r, dsg.E4M3, s, q, None, am)
        return h, y, q, r, am

    whole = run(0, rows)
    parts = [run(a, a + part) for a in range(0, rows, part)]
    for i in range(4):
        assert torch.equal(whole[i], torch.cat([p[i] for p in parts]))
    assert torch.equal(whole[4], torch.stack([p[4] for p in parts]).max(0).values)
