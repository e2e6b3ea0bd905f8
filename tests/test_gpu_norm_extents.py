"""RMSNorm at extents where a grid or a chain of additions would pass its limit.

Tolerances with u = 2^-24: sums of squares over a row of any length are added in 64 bits by a
lane and joined by 6 + 16 fp32 additions, so they are off by at most 24 u, r by half of that and
3 u for the division, root and reciprocal (17 u with 2 to spare), y by 2 u more.  The dot product
of the backward pass: 3 u in each term, 24 u in the sum, 2 u in the mean, and 5 u in what is made
of it: 34 u of the absolute terms."""

import pytest

torch = pytest.importorskip("torch")

import delayed_scaling_gemm_amd as dsg  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0**-24
EPS = 1e-5
BF, F32, U8 = torch.bfloat16, torch.float32, torch.uint8


def rand(g, *shape):
    return torch.randn(shape, generator=g, device=DEV)


@pytest.mark.parametrize("cols", [1, 4, 7])
def test_more_rows_than_a_grid_of_a_row_each(cols):
    rows = (1 << 22) + 33  # of 1024 threads: 2^32 and more
    g = torch.Generator(device=DEV).manual_seed(cols)
    x, gamma = rand(g, rows, cols), rand(g, cols)
    y, r = torch.empty_like(x), torch.empty(rows, device=DEV)
    q, am = torch.empty(rows, cols, dtype=U8, device=DEV), torch.zeros(1, device=DEV)
    used, sat = torch.zeros(1, device=DEV), torch.zeros(1, dtype=torch.int64, device=DEV)
    s = torch.full((1,), 256.0, device=DEV)
    dsg.fp8ds_rmsnorm(x, gamma, EPS, y=y, rstd=r, scale=s, q=q, scale_used=used, amax=am, sat_count=sat)
    torch.cuda.synchronize()
    want = 1.0 / torch.sqrt(x.double().square().mean(1) + EPS)
    assert bool(((r.double() - want).abs() <= 17 * U * want).all())
    yw = x.double() * want[:, None] * gamma.double()
    assert bool(((y.double() - yw).abs() <= 19 * U * yw.abs()).all())
    # the codes and what is combined over all rows, from the y that the call stored
    ys = y * s
    assert torch.equal(q, ys.clamp(-448, 448).to(torch.float8_e4m3fn).view(U8))
    assert float(am) == float(y.abs().max()) and float(used) == 256.0
    assert int(sat) == int((ys.abs() > 448).sum())
    rs, ra = torch.empty(rows, device=DEV), torch.empty(rows, device=DEV)
    dsg.fp8ds_rmsnorm_rowwise(x, gamma, EPS, dsg.E4M3, 0, q, rs, amax=ra)
    torch.cuda.synchronize()
    assert torch.equal(ra, y.abs().amax(1))
    # (a quotient of fp32 numbers taken in fp64 rounds to the fp32 quotient)
    assert torch.equal(rs, torch.where(ra > 0, (448.0 / ra.double()).float(), torch.ones_like(ra)))
    assert torch.equal(q, (y * rs[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(U8))


def test_many_long_rows():
    """Rows longer than the registers, more of them than workgroups, one by one the same."""
    rows, cols = 1200, 32776
    g = torch.Generator(device=DEV).manual_seed(5)
    x, res = rand(g, rows, cols).to(BF), rand(g, rows, cols).to(BF)
    gamma, s = rand(g, cols).to(BF), torch.full((1,), 8.0, device=DEV)

    def run(a, b):
        n = b - a
        h, q = torch.empty(n, cols, dtype=BF, device=DEV), torch.empty(n, cols, dtype=U8, device=DEV)
        qr, rs, am = torch.empty_like(q), torch.empty(n, device=DEV), torch.zeros(1, device=DEV)
        dsg.fp8ds_rmsnorm(x[a:b], gamma, EPS, res[a:b], h, scale=s, q=q, amax=am)
        dsg.fp8ds_rmsnorm_rowwise(x[a:b], gamma, EPS, dsg.E5M2, 0, qr, rs, residual=res[a:b])
        return h, q, qr, rs, am

    whole, parts = run(0, rows), [run(a, a + 100) for a in range(0, rows, 100)]
    for i in range(4):
        assert torch.equal(whole[i], torch.cat([p[i] for p in parts]))
    assert torch.equal(whole[4], torch.stack([p[4] for p in parts]).max(0).values)
    c32 = cols // 32 * 32
    q = torch.empty(rows, c32, dtype=U8, device=DEV)
    sc = torch.empty(rows, c32 // 32, dtype=U8, device=DEV)
    q1, sc1 = torch.empty_like(q), torch.empty_like(sc)
    xc = x[:, :c32].contiguous()
    dsg.fp8ds_rmsnorm_mx(xc, gamma[:c32], EPS, dsg.E4M3, q, sc)
    for a in range(0, rows, 100):
        dsg.fp8ds_rmsnorm_mx(xc[a:a + 100], gamma[:c32], EPS, dsg.E4M3, q1[a:a + 100], sc1[a:a + 100])
    torch.cuda.synchronize()
    assert torch.equal(q, q1) and torch.equal(sc, sc1)


def test_backward_of_a_row_of_2_28_columns():
    """dgamma's join takes 32 columns a workgroup of 512: 2^32 threads and more."""
    cols = (1 << 28) + 40
    g = torch.Generator(device=DEV).manual_seed(4)
    h, dy = rand(g, 1, cols).to(BF), rand(g, 1, cols).to(BF)
    gamma, r = torch.ones(cols, dtype=BF, device=DEV), torch.full((1,), 0.5, device=DEV)
    dx, dg = torch.empty_like(h), torch.full((cols,), 7.0, device=DEV)
    ws = torch.empty(dsg.fp8ds_rmsnorm_bwd_workspace(1, cols), dtype=U8, device=DEV)
    dsg.fp8ds_rmsnorm_bwd(dy, h, r, gamma, dx, dg, ws)
    torch.cuda.synchronize()
    assert torch.equal(dg, (dy.float() * (h.float() * 0.5))[0])


def test_sums_over_very_long_rows():
    """Equal elements: rounded one after the other their squares would drift."""
    rows, cols = 3, 1 << 22
    x = torch.tensor([1.1, 0.3, 0.007], device=DEV)[:, None].expand(rows, cols).contiguous()
    gamma, r = torch.ones(cols, device=DEV), torch.empty(rows, device=DEV)
    y = torch.empty_like(x)
    dsg.fp8ds_rmsnorm(x, gamma, EPS, y=y, rstd=r)
    want = 1.0 / torch.sqrt(x.double().square().mean(1) + EPS)
    torch.cuda.synchronize()
    assert bool(((r.double() - want).abs() <= 17 * U * want).all())
    g = torch.Generator(device=DEV).manual_seed(3)
    dy = 1.0 + 0.1 * rand(g, rows, cols)
    dx, dg = torch.empty_like(x), torch.empty(cols, device=DEV)
    ws = torch.empty(dsg.fp8ds_rmsnorm_bwd_workspace(rows, cols), dtype=U8, device=DEV)
    dsg.fp8ds_rmsnorm_bwd(dy, x, r, gamma, dx, dg, ws)
    torch.cuda.synchronize()
    rd = r.double()[:, None]
    xh = x.double() * rd
    mean = (dy.double() * xh).mean(1, keepdim=True)
    ex = rd * (dy.double() - xh * mean)
    terms = rd * (dy.double().abs() + xh.abs() * (dy.double() * xh).abs().mean(1, keepdim=True))
    assert bool(((dx.double() - ex).abs() <= 34 * U * terms).all())
