"""The gated backward product's FP8 instruction in every shape of tile; tolerances as test_gpu_gated's."""

import pytest

torch = pytest.importorskip("torch")

import delayed_scaling_gemm_amd as dsg  # noqa: E402
import test_gpu_gated as base  # noqa: E402

pytestmark = pytest.mark.gpu


# 256 x 256 tiles whole and with edges; 128 x 128 in two halves of K, alone, and through registers
@pytest.mark.parametrize("fdy", [dsg.E5M2, dsg.E4M3])
@pytest.mark.parametrize("M,F,H", [(4096, 4096, 2048), (3900, 4112, 2176), (300, 272, 2048), (300, 272, 640),
                                   (300, 277, 1000)])
def test_backward_fp8_instruction(M, F, H, fdy):
    base.check_backward(M, F, H, dsg.ACT_SILU, fdy=fdy, fmt=fdy, mma=dsg.MMA_FP8, rel=2.0 ** -9)


@pytest.mark.parametrize("M,F,K", [(3900, 2192, 2176), (300, 144, 2048), (300, 133, 2048)])
def test_forward_fp8_instruction(M, F, K):
    base.check_forward(M, F, K, dsg.ACT_GELU, mma=dsg.MMA_FP8, rel=2.0 ** -10 + 1e-5)
