"""Up to 16 rows of the gated products run exact whatever datapath is named: the same bits."""

import pytest

torch = pytest.importorskip("torch")

import delayed_scaling_gemm_amd as dsg  # noqa: E402
import test_gpu_gated as base  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda"


def generator():
    return torch.Generator(device=DEV).manual_seed(17)


@pytest.mark.parametrize("M,F,H", [(1, 64, 1024), (16, 48, 2048), (7, 33, 1000)])
def test_backward(M, F, H):
    g = generator()
    dy, w = base.codes(g, M, H, 4.0, dsg.E5M2, tails=True), base.codes(g, F, H, 40.0)
    gu = torch.randn(M, 2 * F, generator=g, device=DEV).to(torch.bfloat16)
    a, b = (torch.empty(M, 2 * F, device=DEV) for _ in range(2))
    for mma, out in ((dsg.MMA_EXACT, a), (dsg.MMA_FP8, b)):
        dsg.fp8ds_gated_gemm_bwd(dy, dsg.E5M2, base.vec(4096.0), w, dsg.E4M3, base.vec(1000.0), dsg.ACT_SILU, gu,
                                 dgu=out, mma=mma)
    assert torch.equal(a, b)


@pytest.mark.parametrize("M", [1, 5, 16])
def test_forward_whose_weights_reach_past_2_to_the_31(M):
    """Rows 2^28 bytes apart: the kernel for few rows, whose offsets are 32 bits, does not take them."""
    F, K, ld = 4, 4096, 1 << 28
    g = generator()
    x, w = base.codes(g, M, K, 16.0), base.codes(g, 2 * F, K, 8.0)
    store = torch.empty((2 * F - 1) * ld + K, dtype=torch.uint8, device=DEV)
    far = store.as_strided((2 * F, K), (ld, 1))
    far.copy_(w)
    sx, sw = base.vec(16.0), base.vec(512.0)
    a, b, c = (torch.empty(M, F, device=DEV) for _ in range(3))
    dsg.fp8ds_gated_gemm(x, dsg.E4M3, sx, far, dsg.E4M3, sw, dsg.ACT_SILU, y=a)
    dsg.fp8ds_gated_gemm(x, dsg.E4M3, sx, far, dsg.E4M3, sw, dsg.ACT_SILU, y=b, mma=dsg.MMA_FP8)
    assert torch.equal(a, b)
    dsg.fp8ds_gated_gemm(x, dsg.E4M3, sx, w, dsg.E4M3, sw, dsg.ACT_SILU, y=c)
    e = base.forward64(x, w, F, sx, sw, dsg.ACT_SILU)
    assert ((a.double() - e[2]).abs() <= e[3]).all() and ((c.double() - e[2]).abs() <= e[3]).all()
