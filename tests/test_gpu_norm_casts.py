"""The norm's quantised outputs are those of the separate casts of its FP32 y (of its FP32 dx), bit
for bit: codes, scales, amax and saturation counts, with infinities, NaN and zeros.  Scales that no
recipe makes (0, infinite, NaN) are held against the oracle's encoder instead."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import delayed_scaling_gemm_amd as dsg  # noqa: E402
from oracle import fp8 as ofp8  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32, U8 = torch.bfloat16, torch.float32, torch.uint8
EPS = 1e-5
INF, NAN = float("inf"), float("nan")
SCALES = [1.0, 37.0, 2.0**-140, 1e-45, 3e38, -2.0]
ODD_SCALES = [0.0, INF, -INF, NAN]


def u8(*shape):
    return torch.full(shape, 9, dtype=U8, device=DEV)


def bits(t):
    return t.view(torch.int32) if t.dtype == F32 else t


def same(a, b):
    """Equal bits, any NaN equal to any other."""
    if a.dtype == F32:
        a, b = a.clone(), b.clone()
        a[a.isnan()], b[b.isnan()] = NAN, NAN
    return torch.equal(bits(a), bits(b))


def check_codes(q, y, s, fmt):
    """q = encode(fl32(y s)), NaN codes of either sign."""
    with np.errstate(all="ignore"):
        v = y.cpu().numpy() * np.float32(s)
    want, got = ofp8.encode(v, fmt), q.cpu().numpy()
    nan = np.isnan(v)
    assert (got[nan] & 0x7F == 0x7F).all() and (got[~nan] == want[~nan]).all(), (fmt, s)


def inputs(rows, cols, seed):
    """Finite rows of many magnitudes, a zero row, a row with an infinity and one with a NaN; gammas
    with zeros, an infinity, a NaN and values that carry y past every format."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn(rows, cols, generator=g, device=DEV)
    x *= torch.exp2(torch.randint(-30, 31, (rows, 1), generator=g, device=DEV).float())
    x[0] = 0.0
    if rows > 3:
        x[1, cols // 2], x[2, cols - 1] = INF, NAN
    gamma = torch.randn(cols, generator=g, device=DEV)
    gamma *= torch.exp2(torch.randint(-20, 21, (cols,), generator=g, device=DEV).float())
    gamma[::5] = 0.0
    gamma[cols // 3], gamma[cols // 2 - 1] = 3e38, 1e-40
    return x, gamma


SHAPES = [(5, 32), (9, 96), (300, 100), (7, 1023), (6, 1024), (40, 4096), (5, 8200), (4, 20480), (4, 33024),
          (4, 32801)]


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("special", [False, True])
def test_forward(rows, cols, special):
    x, gamma = inputs(rows, cols, rows + cols)
    if special:
        gamma[cols // 4], gamma[cols // 5] = INF, NAN
    y = torch.empty_like(x)
    dsg.fp8ds_rmsnorm(x, gamma, EPS, y=y)
    for fmt in (dsg.E4M3, dsg.E5M2):
        for s in SCALES:
            sc = torch.full((1,), s, device=DEV)
            out = []
            for fused in (True, False):
                q, su = u8(rows, cols), torch.zeros(1, device=DEV)
                am, sat = torch.zeros(1, device=DEV), torch.zeros(1, dtype=torch.int64, device=DEV)
                if fused:
                    dsg.fp8ds_rmsnorm(x, gamma, EPS, fmt=fmt, scale=sc, q=q, scale_used=su, amax=am,
                                      sat_count=sat)
                else:
                    dsg.fp8ds_cast_acc(y, fmt, sc, q, None, su, am, sat)
                out.append((q, am, sat, su))
            for name, a, b in zip(("q", "amax", "sat", "used"), *out):
                assert same(a, b), (fmt, s, name)
        for s in ODD_SCALES:
            q = u8(rows, cols)
            dsg.fp8ds_rmsnorm(x, gamma, EPS, fmt=fmt, scale=torch.full((1,), s, device=DEV), q=q)
            check_codes(q, y, s, fmt)
        for margin in (0, 3, -2):
            out = []
            for fused in (True, False):
                q, rs, ri, ra = u8(rows, cols), *(torch.zeros(rows, device=DEV) for _ in range(3))
                if fused:
                    dsg.fp8ds_rmsnorm_rowwise(x, gamma, EPS, fmt, margin, q, rs, ri, ra)
                else:
                    dsg.fp8ds_cast_rowwise(y, fmt, margin, q, rs, ri, ra)
                out.append((q, rs, ri, ra))
            for name, a, b in zip(("q", "scale", "inv", "amax"), *out):
                assert same(a, b), (fmt, margin, name)
    if cols % 32 == 0:
        for fmt in (dsg.E4M3, dsg.E5M2, dsg.E2M1):
            w = cols // 2 if fmt == dsg.E2M1 else cols
            q, s, q2, s2 = u8(rows, w), u8(rows, cols // 32), u8(rows, w), u8(rows, cols // 32)
            dsg.fp8ds_rmsnorm_mx(x, gamma, EPS, fmt, q, s)
            if fmt == dsg.E2M1:
                dsg.fp8ds_cast_mxfp4(y, q2, s2)
            else:
                dsg.fp8ds_cast_mx(y, fmt, q2, s2)
            assert torch.equal(s, s2) and torch.equal(q, q2), fmt


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("with_dres", [False, True])
def test_backward(rows, cols, with_dres):
    h, gamma = inputs(rows, cols, 2 * rows + cols)
    dy, _ = inputs(rows, cols, 3 * rows + cols)
    dres = inputs(rows, cols, 5 * rows + cols)[0] if with_dres else None
    r, ws = torch.empty(rows, device=DEV), u8(dsg.fp8ds_rmsnorm_bwd_workspace(rows, cols))
    dsg.fp8ds_rmsnorm(h, gamma, EPS, rstd=r)
    dx, dg = torch.empty_like(h), torch.empty(cols, device=DEV)
    for fmt in (dsg.E4M3, dsg.E5M2):
        for s in SCALES:
            sc = torch.full((1,), s, device=DEV)
            q, su, am = u8(rows, cols), torch.zeros(1, device=DEV), torch.zeros(1, device=DEV)
            sat = torch.zeros(1, dtype=torch.int64, device=DEV)
            dsg.fp8ds_rmsnorm_bwd(dy, h, r, gamma, dx, dg, ws, dres, fmt, sc, q, su, am, sat)
            q2, su2, am2 = u8(rows, cols), torch.zeros(1, device=DEV), torch.zeros(1, device=DEV)
            sat2 = torch.zeros(1, dtype=torch.int64, device=DEV)
            dsg.fp8ds_cast_acc(dx, fmt, sc, q2, None, su2, am2, sat2)
            for name, a, b in (("q", q, q2), ("amax", am, am2), ("sat", sat, sat2), ("used", su, su2)):
                assert same(a, b), (fmt, s, name)
        for s in ODD_SCALES:
            sc, q = torch.full((1,), s, device=DEV), u8(rows, cols)
            dsg.fp8ds_rmsnorm_bwd(dy, h, r, gamma, dx, dg, ws, dres, fmt, sc, q)
            check_codes(q, dx, s, fmt)
