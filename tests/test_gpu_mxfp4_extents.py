"""MXFP4 calls with more rows or columns than one grid of their kernels takes."""

import pytest

torch = pytest.importorskip("torch")

import delayed_scaling_gemm_amd as dsg  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda"
U8 = torch.uint8


def operand(rows, seed):
    """Codes [rows, 16] and scale codes [rows, 1] of +-1 or +-2 times 1 or 2."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    q = torch.empty(rows, 16, dtype=U8, device=DEV)
    for i in range(0, rows, 1 << 25):
        r = torch.randint(0, 256, q[i:i + (1 << 25)].shape, generator=g, device=DEV, dtype=U8)
        q[i:i + (1 << 25)] = (r & 0xCC) | 0x22  # codes 2, 6 and their negatives: 1 and 4
    return q, torch.randint(127, 129, (rows, 1), generator=g, device=DEV, dtype=U8)


def values(q, s):
    c = torch.stack([q & 15, q >> 4], -1).reshape(q.shape[0], 32)
    v = torch.where(c & 4 > 0, 4.0, 1.0) * torch.where(c & 8 > 0, -1.0, 1.0)
    return v * torch.exp2(s.float() - 127)


@pytest.mark.parametrize("M,N,ldb", [(65535 * 32 + 45, 1, 1 << 21), (65535 * 64, 1, 1 << 21),
                                     (3, (1 << 29) + 70, 32)])
def test_product_beyond_one_grid(M, N, ldb):
    """Whole numbers of at most 32 x 8 x 8: exact sums, and one rounding to BF16 on both sides."""
    (a, sa), (b, sb) = operand(M, 1), operand(N, 2)
    am = torch.zeros(1, device=DEV)
    c = torch.full((M, N), 9.0, dtype=torch.bfloat16, device=DEV)
    dsg.fp8ds_gemm_mxfp4(M, N, 32, a, dsg.E2M1, 32, sa, 1, b, ldb, sb, 1, c, N, am)
    torch.cuda.synchronize()
    top = 0.0
    for i in range(0, max(M, N), 1 << 24):
        ms, ns = (slice(i, i + (1 << 24)), slice(None)) if M > N else (slice(None), slice(i, i + (1 << 24)))
        want = (values(a[ms], sa[ms]) @ values(b[ns], sb[ns]).t()).bfloat16()
        assert torch.equal(c[ms, ns], want)
        top = max(top, float(want.abs().max()))
    assert float(am) == top
