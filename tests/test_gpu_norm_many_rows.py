"""RMSNorm with more rows than one round of its workgroups: every variant goes on to further
rows, with a partial last round, and gives what it gives for a few rows at a time.

The forward grid is at most 8 workgroups per CU of 256 / TPR rows each (TPR threads a row, 16 to
256), one per CU of one row where 1024 threads take it; the backward grid at most 1024 workgroups.
`rounds` states those rules again, and the tests assert that they are passed."""

import pytest

torch = pytest.importorskip("torch")

import delayed_scaling_gemm_amd as dsg  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32, U8 = torch.bfloat16, torch.float32, torch.uint8
EPS = 1e-5
U = 2.0**-24


def tpr(cols):
    g = -(-cols // 8)
    return 16 if g <= 16 else 64 if g <= 128 else 256 if g <= 1024 else 1024


def rounds(rows, cols, backward=False):
    cus = torch.cuda.get_device_properties(0).multi_processor_count
    t = tpr(cols)
    if backward:
        per = 1024 * (256 // t if t <= 256 else 1)
    else:
        per = 8 * cus * (256 // t) if t <= 256 else cus
    return rows / per


def inputs(rows, cols, xt, ht, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn(rows, cols, generator=g, device=DEV).to(xt)
    res = torch.randn(rows, cols, generator=g, device=DEV).mul_(2).to(ht)
    gamma = (1 + 0.2 * torch.randn(cols, generator=g, device=DEV)).to(xt)
    return x, res, gamma


SHAPES = [(70001, 100), (70001, 96), (17003, 500), (17003, 512), (17003, 1000), (17003, 1023),
          (17003, 1024), (5003, 2047), (5003, 2048), (5003, 4095), (5003, 4096), (4099, 8191),
          (4099, 8192), (600, 16383), (600, 16384)]


@pytest.mark.parametrize("xt,ht", [(BF, BF), (BF, F32), (F32, F32)])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_forward(rows, cols, xt, ht):
    assert rounds(rows, cols) > 2
    x, res, gamma = inputs(rows, cols, xt, ht, rows + cols)
    s = torch.full((1,), 300.0, device=DEV)
    few = max(1, int(rows / rounds(rows, cols)))  # rows that one round takes

    def run(a, b, r):
        n = b - a
        h, y = r.clone(), torch.empty(n, cols, dtype=xt, device=DEV)
        q, qr = (torch.empty(n, cols, dtype=U8, device=DEV) for _ in range(2))
        rstd, rs, ra = (torch.empty(n, device=DEV) for _ in range(3))
        am, sat = torch.zeros(1, device=DEV), torch.zeros(1, dtype=torch.int64, device=DEV)
        # the residual stream in place
        dsg.fp8ds_rmsnorm(x[a:b], gamma, EPS, h, h, y, rstd, dsg.E4M3, s, q, None, am, sat)
        dsg.fp8ds_rmsnorm_rowwise(x[a:b], gamma, EPS, dsg.E5M2, 1, qr, rs, amax=ra, residual=r)
        out = [h, y, rstd, q, qr, rs, ra]
        if cols % 32 == 0:
            for fmt, w in ((dsg.E4M3, cols), (dsg.E2M1, cols // 2)):
                m, ms = (torch.empty(n, k, dtype=U8, device=DEV) for k in (w, cols // 32))
                dsg.fp8ds_rmsnorm_mx(x[a:b], gamma, EPS, fmt, m, ms, residual=r)
                out += [m, ms]
        return out, am, sat

    whole, am, sat = run(0, rows, res)
    top, count = 0.0, 0
    for at in range(0, rows, few):
        end = min(rows, at + few)
        part, pam, psat = run(at, end, res[at:end])
        for i, (a, b) in enumerate(zip(whole, part)):
            assert torch.equal(a[at:end], b), (i, at)
        top, count = max(top, float(pam)), count + int(psat)
    assert float(am) == top and int(sat) == count
    # and against the formula
    h = (x.float() + res.float()).to(ht).double()
    want = 1 / torch.sqrt(h.square().mean(1) + EPS)
    assert torch.equal(whole[0].double(), h)
    assert bool(((whole[2].double() - want).abs() <= 52 * U * want).all())
    yw = h * want[:, None] * gamma.double()
    half = 2.0**-8 if xt == BF else U
    assert bool(((whole[1].double() - yw).abs() <= (54 * U + half) * yw.abs() * 1.01).all())


BWD = [(40001, 100), (40001, 96), (9001, 500), (9001, 512), (9001, 1001), (3001, 2047), (3001, 2048),
       (2500, 4096), (2500, 8191), (2500, 8192), (2500, 9000), (2500, 16384)]


@pytest.mark.parametrize("xt,ht", [(BF, BF), (BF, F32), (F32, F32)])
@pytest.mark.parametrize("rows,cols", BWD)
def test_backward(rows, cols, xt, ht):
    if cols <= 8192:
        assert rounds(rows, cols, True) > 2
    x, h, gamma = inputs(rows, cols, xt, ht, rows + 3 * cols)
    dy = x
    r = (1 / torch.sqrt(h.double().square().mean(1) + EPS)).float()
    s = torch.full((1,), 200.0, device=DEV)

    def run(a, b, dres):
        n = b - a
        ws = torch.full((max(16, dsg.fp8ds_rmsnorm_bwd_workspace(n, cols)),), 255, dtype=U8, device=DEV)
        dx, q = torch.empty(n, cols, dtype=ht, device=DEV), torch.empty(n, cols, dtype=U8, device=DEV)
        dg, am = torch.empty(cols, device=DEV), torch.zeros(1, device=DEV)
        sat = torch.zeros(1, dtype=torch.int64, device=DEV)
        if dres is not None:
            dx.copy_(dres[a:b])  # in place
        dsg.fp8ds_rmsnorm_bwd(dy[a:b], h[a:b], r[a:b], gamma, dx, dg, ws, dx if dres is not None else None,
                              dsg.E5M2, s, q, None, am, sat)
        return dx, q, dg, am, sat

    for dres in (None, h):
        dx, q, dg, am, sat = run(0, rows, dres)
        few, top, count = 900, 0.0, 0
        for at in range(0, rows, few):
            end = min(rows, at + few)
            p = run(at, end, dres)
            assert torch.equal(dx[at:end], p[0]) and torch.equal(q[at:end], p[1]), at
            top, count = max(top, float(p[3])), count + int(p[4])
        assert float(am) == top and int(sat) == count
        # dgamma: (rows that a workgroup adds + 70) u of the absolute sum, 4 u in a term
        xh = h.double() * r.double()[:, None]
        want, mag = (dy.double() * xh).sum(0), (dy.double() * xh).abs().sum(0)
        chain = rounds(rows, cols, True) if cols <= 8192 else rows / 1024
        assert bool(((dg.double() - want).abs() <= (chain + 75) * U * mag).all())
