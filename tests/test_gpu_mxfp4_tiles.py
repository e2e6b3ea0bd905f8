"""MXFP4 products on the tile kernels: both tile sizes, every format of A on each of its datapaths,
both layouts of the scale codes, odd and even numbers of stages.

The shapes are chosen by the launcher's rule, stated again in `kernel`: the tests assert which
kernel they reach.  K, in stages of 256 (FP4 x FP4, two buffers) or 128 (FP8 A, three): 32, 96 and
160 end inside the first; the others give 1 to 9 of them, odd and even, with every remainder of 3.
Codes are read 16 at a time from K = 512 on where K / 32 and the rows of codes are at dwords,
else (K below, 1056, odd addresses) a dword or two a stage.

Whole numbers: elements of 0, 1, 2, 3, 4 and scales of 1 and 2, so products reach 64 and sums
64 x 1152 < 2^17: exact in FP32 (and in the FP8 instruction's 13 bits below a group's largest
product, 64 = 2^6).  Results have to be equal, BF16 ones after one rounding.

Random operands on v_mfma_scale_f32_32x32x64: two blocks and the accumulator, each off by less
than a unit of 2^-23 of the largest; ceil(K / 64) + 1 instructions (the loop starts with one of
zeros): (3 (K / 64 + 2)) 2^-23 sum |ab|.  The FP8 datapath's groups of 8: 8 x 2^-13 of each group's
largest.  The exact datapath: K + 16 additions of a unit of 2^-23."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import delayed_scaling_gemm_amd as dsg  # noqa: E402
from oracle import mx as omx  # noqa: E402
from oracle import mxfp4 as o4  # noqa: E402
from tests.parity import FP8_GROUP, FP8_GROUP_UNIT, bf16_ulp, fp8_group_max_sum  # noqa: E402
from tests.test_gpu_gemm import finite_codes  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda"
U8 = torch.uint8
E2M1, E4M3, E5M2 = dsg.E2M1, dsg.E4M3, dsg.E5M2
EXACT, FP8 = dsg.MMA_EXACT, dsg.MMA_FP8
PATHS = [(E2M1, EXACT), (E4M3, EXACT), (E4M3, FP8), (E5M2, EXACT), (E5M2, FP8)]
KS = [32, 96, 160, 288, 480, 512, 640, 768, 896, 1024, 1056, 1152]


def kernel(M, N):
    """256 or 128: the tiles that a product of these rows and columns takes, else 0."""
    cus = torch.cuda.get_device_properties(0).multi_processor_count
    if M <= 16 or -(-M // 32) * -(-N // 32) <= 2 * cus:
        return 0
    return 256 if -(-M // 256) * -(-N // 256) >= cus else 128


SIZES = {128: (1000, 1100), 256: (4100, 4000)}


def test_the_sizes_reach_the_kernels():
    for tile, (M, N) in SIZES.items():
        assert kernel(M, N) == tile


# codes of 0, 1, 2, 3, 4 and -1 .. -4 in each format
WHOLE = {E2M1: [0, 2, 4, 5, 6, 10, 12, 13, 14],
         E4M3: [0x00, 0x38, 0x40, 0x44, 0x48, 0xB8, 0xC0, 0xC4, 0xC8],
         E5M2: [0x00, 0x3C, 0x40, 0x42, 0x44, 0xBC, 0xC0, 0xC2, 0xC4]}
NUMBERS = [0.0, 1.0, 2.0, 3.0, 4.0, -1.0, -2.0, -3.0, -4.0]


def whole(rows, K, fmt, seed):
    """(codes, scale codes, values) of whole numbers."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    i = torch.randint(0, 9, (rows, K), generator=g, device=DEV)
    c = torch.tensor(WHOLE[fmt], dtype=U8, device=DEV)[i]
    if fmt == E2M1:
        c = c[:, 0::2] | (c[:, 1::2] << 4)
    s = torch.randint(127, 129, (rows, K // 32), generator=g, device=DEV, dtype=U8)
    v = torch.tensor(NUMBERS, device=DEV)[i] * (s.float() - 126).repeat_interleave(32, 1)
    return c.contiguous(), s, v


def placed(t, width, offset, fill):
    """t's rows in rows of `width` bytes from byte `offset` on, `fill` around them."""
    w = torch.full((t.shape[0], width), fill, dtype=U8, device=DEV)
    w[:, offset:offset + t.shape[1]] = t
    return w[:, offset:]


@pytest.mark.parametrize("tile", [128, 256])
@pytest.mark.parametrize("fa,mma", PATHS)
@pytest.mark.parametrize("K", KS)
def test_whole_numbers(tile, fa, mma, K):
    M, N = SIZES[tile]
    pa = 2 if fa == E2M1 else 1
    a, sa, av = whole(M, K, fa, K + fa)
    b, sb, bv = whole(N, K, E2M1, K + 7)
    want = av @ bv.t()  # (whole numbers: exact in fp32)
    nb = K // 32
    # codes of rows as they come; apart and at odd addresses, NaN codes and NaN or largest
    # elements next to each row's last
    for wide in (False, True):
        if wide:
            args = (placed(a, (K + 64) // pa, 0, 0x7F), fa, K + 64, placed(sa, nb + 6, 3, 255), nb + 6,
                    placed(b, (K + 96) // 2, 16, 0x77), K + 96, placed(sb, nb + 5, 1, 255), nb + 5)
        else:
            args = (a, fa, K, sa, nb, b, K, sb, nb)
        am = torch.full((1,), 1e9, device=DEV)
        c = torch.full((M, N), 0.5, device=DEV)
        dsg.fp8ds_gemm_mxfp4(M, N, K, *args, c, N, am, mma=mma)
        torch.cuda.synchronize()
        assert torch.equal(c, want), wide
        assert float(am) == float(want.abs().max())
        # BF16, rows that are not at 16 bytes, untouched past N
        c = torch.full((M, N + 3), 0.5, dtype=torch.bfloat16, device=DEV)
        dsg.fp8ds_gemm_mxfp4(M, N, K, *args, c, N + 3, am, mma=mma)
        c2 = torch.full((M, N), 0.5, dtype=torch.bfloat16, device=DEV)
        dsg.fp8ds_gemm_mxfp4(M, N, K, *args, c2, N, None, mma=mma)
        torch.cuda.synchronize()
        assert torch.equal(c[:, :N], want.bfloat16()) and bool((c[:, N:] == 0.5).all()), wide
        assert torch.equal(c2, want.bfloat16())
        assert float(am) == float(want.bfloat16().float().abs().max())


@pytest.mark.parametrize("tile", [128, 256])
@pytest.mark.parametrize("fa,mma", PATHS)
@pytest.mark.parametrize("K", [288, 896, 1056])
def test_random_operands(tile, fa, mma, K):
    M, N = SIZES[tile]
    rng = np.random.default_rng(tile + K + fa)
    sa = rng.integers(122, 131, (M, K // 32)).astype(np.uint8)
    sb = rng.integers(122, 131, (N, K // 32)).astype(np.uint8)
    b = rng.integers(0, 256, (N, K // 2)).astype(np.uint8)
    if fa == E2M1:
        a = rng.integers(0, 256, (M, K // 2)).astype(np.uint8)
        av = o4.dequant(a, sa)
    else:
        a = finite_codes(rng, (M, K), fa)
        av = omx.mx_dequant(a, sa, fa)
    bv = o4.dequant(b, sb)
    c = torch.empty(M, N, device=DEV)
    dev = [torch.from_numpy(t).to(DEV) for t in (a, sa, b, sb)]
    dsg.fp8ds_gemm_mxfp4(M, N, K, dev[0], fa, K, dev[1], K // 32, dev[2], K, dev[3], K // 32, c, N,
                         mma=mma)
    torch.cuda.synchronize()
    ad, bd = torch.from_numpy(av).to(DEV), torch.from_numpy(bv).to(DEV)
    want, mag = ad @ bd.t(), ad.abs() @ bd.abs().t()
    if fa == E2M1 or mma == FP8:
        bound = 3 * (K / 64 + 2) * 2.0**-23 * mag
    else:
        bound = (K + 16) * 2.0**-23 * mag
    err = (c.double() - want).abs()
    if fa != E2M1 and mma == FP8:  # the groups' bound, on rows of every tile and both edges
        rows = np.unique(np.r_[0, np.arange(37, M, 211), M - 1])
        groups = FP8_GROUP * FP8_GROUP_UNIT * fp8_group_max_sum(av[rows], bv.T)
        assert bool((err[rows] <= bound[rows] + torch.from_numpy(groups).to(DEV)).all())
    else:
        assert bool((err <= bound).all())


@pytest.mark.parametrize("tile", [128, 256])
@pytest.mark.parametrize("fa,mma", PATHS)
@pytest.mark.parametrize("K", [160, 640])
def test_nan_blocks(tile, fa, mma, K):
    M, N = SIZES[tile]
    a, sa, av = whole(M, K, fa, 3 * K)
    b, sb, bv = whole(N, K, E2M1, 5 * K)
    rows, cols = [0, 300, M - 1], [5, 129, N - 1]
    for i, r in enumerate(rows):
        sa[r, (i * 2) % (K // 32)] = 255
    for i, n in enumerate(cols):
        sb[n, (K // 32 - 1 - i)] = 255
    want = av @ bv.t()
    want[rows], want[:, cols] = float("nan"), float("nan")
    c = torch.empty(M, N, device=DEV)
    dsg.fp8ds_gemm_mxfp4(M, N, K, a, fa, K, sa, K // 32, b, K, sb, K // 32, c, N, mma=mma)
    torch.cuda.synchronize()
    assert torch.equal(c.isnan(), want.isnan())
    assert torch.equal(c.nan_to_num(0.0), want.nan_to_num(0.0))


@pytest.mark.parametrize("fa,mma", PATHS)
def test_edges_of_the_tiles(fa, mma):
    """Row and column counts around the tiles' borders, and few of one with many of the other."""
    for M, N in ((17, 17000), (33, 9000), (16900, 33), (129, 5000), (1025, 1023), (255, 2400)):
        assert kernel(M, N) == 128, (M, N)
        a, sa, av = whole(M, 544, fa, M)
        b, sb, bv = whole(N, 544, E2M1, N)
        c = torch.empty(M, N, dtype=torch.bfloat16, device=DEV)
        dsg.fp8ds_gemm_mxfp4(M, N, 544, a, fa, 544, sa, 17, b, 544, sb, 17, c, N, mma=mma)
        torch.cuda.synchronize()
        assert torch.equal(c, (av @ bv.t()).bfloat16()), (M, N)
    for M, N in ((4097, 4095), (16129, 1025), (257, 65281)):
        assert kernel(M, N) == 256, (M, N)
        a, sa, av = whole(M, 544, fa, M)
        b, sb, bv = whole(N, 544, E2M1, N)
        c = torch.empty(M, N, device=DEV)
        dsg.fp8ds_gemm_mxfp4(M, N, 544, a, fa, 544, sa, 17, b, 544, sb, 17, c, N, mma=mma)
        torch.cuda.synchronize()
        assert torch.equal(c, av @ bv.t()), (M, N)


def test_rows_far_apart_take_the_direct_kernel():
    """From 2^21 elements between rows on, the tiles' 31-bit offsets would not reach them."""
    M, N, K, ld = 40, 1100, 96, 1 << 21
    a, sa, av = whole(M, K, E2M1, 1)
    b, sb, bv = whole(N, K, E2M1, 2)
    A = torch.full((M, ld // 2), 0x77, dtype=U8, device=DEV)
    A[:, :K // 2] = a
    c = torch.empty(M, N, device=DEV)
    dsg.fp8ds_gemm_mxfp4(M, N, K, A, E2M1, ld, sa, K // 32, b, K, sb, K // 32, c, N)
    torch.cuda.synchronize()
    assert torch.equal(c, av @ bv.t())


def test_empty_k_and_the_linear_step_on_tiles():
    for tile, (M, N) in SIZES.items():
        one = torch.zeros(max(M, N), 16, dtype=U8, device=DEV)
        c = torch.full((M, N), 3.0, dtype=torch.bfloat16, device=DEV)
        am = torch.full((1,), 3.0, device=DEV)
        dsg.fp8ds_gemm_mxfp4(M, N, 0, one, E2M1, 32, one, 1, one, 32, one, 1, c, N, am)
        torch.cuda.synchronize()
        assert bool((c == 0).all()) and float(am) == 0.0
    from delayed_scaling_gemm_amd.linear import MXFP4Linear

    M, K, N = 4096, 4064, 4128  # all three products on tiles of 256
    g = torch.Generator(device=DEV).manual_seed(0)
    x, w, dy = (torch.randn(s, generator=g, device=DEV).mul_(m).bfloat16()
                for s, m in (((M, K), 1.0), ((K, N), 0.02), ((M, N), 1e-3)))
    out = MXFP4Linear(device=DEV).step(x, w, dy)
    torch.cuda.synchronize()
    q = lambda t: torch.from_numpy(o4.dequant(*o4.cast(t.float().cpu().numpy()))).to(DEV)  # noqa: E731
    xf, wf, df = q(x), q(w), q(dy)
    xt, wt, dt = q(x.t().contiguous()), q(w.t().contiguous()), q(dy.t().contiguous())
    for name, a, b in (("y", xf, wt), ("dx", df, wf), ("dw", xt, dt)):
        assert kernel(a.shape[0], b.shape[0]) == 256
        want, k = a @ b.t(), a.shape[1]
        bound = 3 * (k / 64 + 2) * 2.0**-23 * (a.abs() @ b.abs().t())
        half = torch.from_numpy(bf16_ulp((want.abs() + bound).cpu().numpy()) / 2).to(DEV)
        assert bool(((out[name].double() - want).abs() <= bound + half).all()), name
