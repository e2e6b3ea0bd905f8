"""GPU parity of MXFP4 against its oracle (oracle/mxfp4.py): casts and values bit for bit,
products within a bound derived from the matrix instruction.

An instruction adds the four blocks of 128 k and the accumulator; each of these five
terms loses less than one unit of 2^-23 of the largest.  With n instructions, and 16
fp32 additions across waves:  |acc - exact| <= (5 n + 16) 2^-23 sum |ab|.  With an FP8
operand the products inside a group of 8 lose 2^-13 of the group's largest each."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import delayed_scaling_gemm_amd as dsg  # noqa: E402
from delayed_scaling_gemm_amd.linear import MXFP4Linear  # noqa: E402
from oracle import bf16 as obf16  # noqa: E402
from oracle import mx as omx  # noqa: E402
from oracle import mxfp4 as o4  # noqa: E402
from tests.parity import FP8_GROUP, FP8_GROUP_UNIT, bf16_bits, bf16_ulp, fp8_group_max_sum  # noqa: E402
from tests.test_gpu_gemm import finite_codes  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda"


def values(rows, cols, seed, bf16, specials=True):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((rows, cols)) * 2.0 ** rng.integers(-30, 31, (rows, 1))
    x[rng.random((rows, cols)) < 0.2] *= 0.25
    # exact ties, and values next to them
    x[:, ::7] = np.sign(x[:, ::7]) * rng.choice([0.25, 0.75, 2.5, 5.0, 6.0, 7.0], x[:, ::7].shape)
    if specials and rows > 6:
        x[0] = 0.0
        x[1, cols // 2] = np.inf
        x[2, 3] = np.nan
        x[3] = 2.0**-130 * rng.standard_normal(cols)
        x[4] = 3e38 * rng.uniform(-1, 1, cols)
        x[5, ::2] = -0.0
    t = torch.from_numpy(x.astype(np.float32))
    if bf16:
        t = t.to(torch.bfloat16)
    return t.to(DEV), t.float().numpy()


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("shape", [(1, 32), (7, 32), (33, 96), (64, 4096), (5, 14336), (257, 160)])
def test_cast_and_values(shape, bf16):
    rows, cols = shape
    x, ref = values(rows, cols, rows + cols, bf16)
    q = torch.empty(rows, cols // 2, dtype=torch.uint8, device=DEV)
    s = torch.empty(rows, cols // 32, dtype=torch.uint8, device=DEV)
    dsg.fp8ds_cast_mxfp4(x, q, s)
    y, y32 = torch.empty(rows, cols, dtype=torch.bfloat16, device=DEV), torch.empty(rows, cols, device=DEV)
    dsg.fp8ds_dequant_mxfp4(q, s, y)
    dsg.fp8ds_dequant_mxfp4(q, s, y32)
    torch.cuda.synchronize()
    oq, os_ = o4.cast(ref)
    np.testing.assert_array_equal(s.cpu().numpy(), os_)
    np.testing.assert_array_equal(q.cpu().numpy(), oq)
    d = o4.dequant(oq, os_)
    np.testing.assert_array_equal(y32.cpu().numpy().astype(np.float64), d)
    np.testing.assert_array_equal(y.float().cpu().numpy().astype(np.float64), d)


def test_cast_every_bf16_pattern():
    """All finite BF16 patterns, 31 beside a fixed largest element in each block, for
    several block exponents."""
    bits = np.arange(65536, dtype=np.uint32)
    v = (bits << 16).view(np.float32)
    v = v[np.isfinite(v)]
    v = np.concatenate([v, np.zeros(-len(v) % 31, np.float32)]).reshape(-1, 31)
    for top in (0.0, 1.0, 1.75, 2.0**-100, 2.0**120):
        x = np.concatenate([np.full((len(v), 1), top, np.float32), v], axis=1)
        t = torch.from_numpy(x).to(torch.bfloat16).to(DEV)
        q = torch.empty(len(v), 16, dtype=torch.uint8, device=DEV)
        s = torch.empty(len(v), 1, dtype=torch.uint8, device=DEV)
        dsg.fp8ds_cast_mxfp4(t, q, s)
        torch.cuda.synchronize()
        oq, os_ = o4.cast(t.float().cpu().numpy())
        np.testing.assert_array_equal(s.cpu().numpy(), os_)
        np.testing.assert_array_equal(q.cpu().numpy(), oq)


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("shape", [(32, 32), (96, 160), (128, 128), (256, 416), (992, 64), (160, 1024)])
def test_cast_transposed_copy(shape, bf16):
    rows, cols = shape
    x, ref = values(rows, cols, 3 * rows + cols, bf16)
    u8 = dict(dtype=torch.uint8, device=DEV)
    q, s = torch.empty(rows, cols // 2, **u8), torch.empty(rows, cols // 32, **u8)
    qt, st = torch.empty(cols, rows // 2, **u8), torch.empty(cols, rows // 32, **u8)
    dsg.fp8ds_cast_mxfp4(x, q, s, qt, st)
    torch.cuda.synchronize()
    oq, os_ = o4.cast(ref)
    oqt, ost = o4.cast(np.ascontiguousarray(ref.T))
    for got, want in ((s, os_), (q, oq), (st, ost), (qt, oqt)):
        np.testing.assert_array_equal(got.cpu().numpy(), want)


# ------------------------------------------------------------------ products


def operand(rng, rows, K, fmt, wide=False):
    sc = rng.integers(100, 150, (rows, K // 32)) if wide else rng.integers(122, 131, (rows, K // 32))
    if fmt == dsg.E2M1:
        c = rng.integers(0, 256, (rows, K // 2)).astype(np.uint8)
        return c, sc.astype(np.uint8), o4.dequant(c, sc)
    c = finite_codes(rng, (rows, K), fmt)
    return c, sc.astype(np.uint8), omx.mx_dequant(c, sc, fmt)


def bound(av, bv, K, fa):
    sa = np.abs(av) @ np.abs(bv).T
    n = -(-K // 128)
    b = (5 * n + 16) * 2.0**-23 * sa
    if fa != dsg.E2M1:
        b = b + FP8_GROUP * FP8_GROUP_UNIT * fp8_group_max_sum(av, bv.T)
    return b


def run_gemm(a, sa, fa, b, sb, K, out=torch.float32, amax=None, ldc=None):
    M, N = a.shape[0], b.shape[0]
    c = torch.full((M, ldc or N), 77.0, dtype=out, device=DEV)
    t = [torch.from_numpy(np.ascontiguousarray(v)).to(DEV) for v in (a, sa, b, sb)]
    dsg.fp8ds_gemm_mxfp4(M, N, K, t[0], fa, max(K, 32), t[1], max(K // 32, 1), t[2], max(K, 32), t[3],
                         max(K // 32, 1), c, ldc or N, amax)
    torch.cuda.synchronize()
    return c


GEMMS = [(1, 1, 32), (1, 4096, 4096), (1, 100, 14336), (2, 64, 96), (13, 130, 160), (16, 257, 1024),
         (17, 64, 512), (33, 70, 128), (64, 64, 416), (100, 300, 256), (129, 127, 96), (200, 520, 1056),
         (300, 256, 64), (512, 384, 640), (31, 8, 4096)]


@pytest.mark.parametrize("fa", [dsg.E2M1, dsg.E4M3, dsg.E5M2])
@pytest.mark.parametrize("shape", GEMMS)
def test_gemm(shape, fa):
    M, N, K = shape
    rng = np.random.default_rng(M + 3 * N + 7 * K + fa)
    a, sa, av = operand(rng, M, K, fa)
    b, sb, bv = operand(rng, N, K, dsg.E2M1)
    acc, bd = av @ bv.T, bound(av, bv, K, fa)
    am = torch.zeros(1, device=DEV)
    c = run_gemm(a, sa, fa, b, sb, K, amax=am)
    assert (np.abs(c.cpu().numpy() - acc) <= bd).all()
    assert float(am) == float(c.abs().max())
    c16 = run_gemm(a, sa, fa, b, sb, K, out=torch.bfloat16, amax=am, ldc=N + 3)
    got = c16[:, :N].float().cpu().numpy()
    assert (np.abs(got - acc) <= bd + bf16_ulp(np.abs(acc) + bd) / 2).all()
    assert (c16[:, N:] == 77).all() and float(am) == np.abs(got).max()


@pytest.mark.parametrize("fa", [dsg.E2M1, dsg.E4M3])
@pytest.mark.parametrize("shape", [(5, 96, 1024), (300, 200, 512)])
def test_gemm_exact_integers(shape, fa):
    """Small whole numbers and scales of 1 and 2: every sum is exact, a wrong block, scale
    or element shows."""
    M, N, K = shape
    rng = np.random.default_rng(K + fa)
    mags = np.array([0, 2, 4, 5, 6])  # codes of 0, 1, 2, 3, 4
    code = lambda r: (mags[rng.integers(0, 5, (r, K))] | (8 * rng.integers(0, 2, (r, K)))).astype(np.uint8)  # noqa: E731
    bc = code(N)
    b, sb = o4.pack(bc), rng.integers(127, 129, (N, K // 32)).astype(np.uint8)
    sa = rng.integers(127, 129, (M, K // 32)).astype(np.uint8)
    if fa == dsg.E2M1:
        a = o4.pack(code(M))
        av = o4.dequant(a, sa)
    else:
        from oracle import fp8 as ofp8
        a = ofp8.encode(rng.integers(-4, 5, (M, K)).astype(np.float32), fa)
        av = omx.mx_dequant(a, sa, fa)
    c = run_gemm(a, sa, fa, b, sb, K)
    np.testing.assert_array_equal(c.cpu().numpy().astype(np.float64), av @ o4.dequant(b, sb).T)


@pytest.mark.parametrize("M", [1, 40, 300])
def test_gemm_wide_scales_nan_blocks_and_empty_k(M):
    rng = np.random.default_rng(M)
    N, K = 72, 512
    a, sa, av = operand(rng, M, K, dsg.E2M1, wide=True)
    b, sb, bv = operand(rng, N, K, dsg.E2M1, wide=True)
    sb[5, 3] = 255
    sa[M - 1, 7] = 255
    av, bv = o4.dequant(a, sa), o4.dequant(b, sb)
    c = run_gemm(a, sa, dsg.E2M1, b, sb, K).cpu().numpy()
    keep = np.ones((M, N), bool)
    keep[:, 5] = keep[M - 1] = False
    assert np.isnan(c[~keep]).all() and np.isfinite(c[keep]).all()
    av, bv = np.nan_to_num(av), np.nan_to_num(bv)
    err, bd = np.abs(c - av @ bv.T), bound(av, bv, K, dsg.E2M1)
    assert (err[keep] <= bd[keep]).all()
    am = torch.full((1,), 3.0, device=DEV)
    z = run_gemm(np.zeros((M, 16), np.uint8), np.zeros((M, 1), np.uint8), dsg.E2M1,
                 np.zeros((N, 16), np.uint8), np.zeros((N, 1), np.uint8), 0, amax=am)
    assert (z == 0).all() and float(am) == 0.0


@pytest.mark.parametrize("fa", [dsg.E2M1, dsg.E4M3])
@pytest.mark.parametrize("M", [3, 150])
def test_gemm_strided_operands(M, fa):
    """Rows and scale rows further apart than they are long (a slice of a wider matrix),
    scale rows at odd addresses."""
    rng = np.random.default_rng(M)
    N, K = 140, 288
    a, sa, av = operand(rng, M, K, fa)
    b, sb, bv = operand(rng, N, K, dsg.E2M1)
    pa = 2 if fa == dsg.E2M1 else 1
    A = torch.full((M, (K + 64) // pa), 0x77, dtype=torch.uint8, device=DEV)
    B = torch.full((N, (K + 96) // 2), 0x77, dtype=torch.uint8, device=DEV)
    SA, SB = (torch.full((n, K // 32 + 2), 255, dtype=torch.uint8, device=DEV) for n in (M, N))
    A[:, :K // pa] = torch.from_numpy(a).to(DEV)
    B[:, 16:16 + K // 2] = torch.from_numpy(b).to(DEV)
    SA[:, 1:1 + K // 32] = torch.from_numpy(sa).to(DEV)
    SB[:, 1:1 + K // 32] = torch.from_numpy(sb).to(DEV)
    c = torch.empty(M, N, device=DEV)
    dsg.fp8ds_gemm_mxfp4(M, N, K, A, fa, K + 64, SA[:, 1:], K // 32 + 2, B[:, 16:], K + 96, SB[:, 1:],
                         K // 32 + 2, c, N)
    torch.cuda.synchronize()
    assert (np.abs(c.cpu().numpy() - av @ bv.T) <= bound(av, bv, K, fa)).all()


def test_linear_step_and_forward():
    M, K, N = 288, 416, 160
    rng = np.random.default_rng(8)
    arr = [rng.standard_normal(s) * m for s, m in (((M, K), 1.0), ((K, N), 0.02), ((M, N), 1e-3))]
    x, w, dy = (torch.from_numpy(a).to(DEV).to(torch.bfloat16) for a in arr)
    layer = MXFP4Linear(device=DEV)
    out = layer.step(x, w, dy)
    torch.cuda.synchronize()
    q = lambda t: o4.dequant(*o4.cast(np.ascontiguousarray(t)))  # noqa: E731
    xf, wf, df = (t.float().cpu().numpy() for t in (x, w, dy))
    for name, a, b in (("y", q(xf), q(wf.T)), ("dx", q(df), q(wf)), ("dw", q(xf.T), q(df.T))):
        acc, bd = a @ b.T, bound(a, b, a.shape[1], dsg.E2M1)
        got = out[name].float().cpu().numpy()
        assert (np.abs(got - acc) <= bd + bf16_ulp(np.abs(acc) + bd) / 2).all(), name
    y = out["y"].clone()
    layer.quantize(w)  # serving: the weights once, then any number of tokens
    for m in (1, 7, M):
        assert torch.equal(layer.forward(x[:m]), y[:m]) or m <= 16
        f8 = layer.forward(x[:m], fmt=dsg.E4M3)
        xe = omx.mx_dequant(*omx.mx_cast(xf[:m], dsg.E4M3), dsg.E4M3)
        b = q(wf.T)
        acc, bd = xe @ b.T, bound(xe, b, K, dsg.E4M3)
        assert (np.abs(f8.float().cpu().numpy() - acc) <= bd + bf16_ulp(np.abs(acc) + bd) / 2).all()


def test_graph_replays():
    x = torch.randn(48, 512, device=DEV, dtype=torch.bfloat16)
    w = torch.randn(512, 96, device=DEV, dtype=torch.bfloat16)
    layer = MXFP4Linear(device=DEV)
    layer.quantize(w)
    layer.forward(x)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = layer.forward(x)
    for _ in range(3):
        x.copy_(torch.randn(48, 512, device=DEV))
        graph.replay()
        torch.cuda.synchronize()
        got = y.clone()
        assert torch.equal(layer.forward(x), got)
