"""What fp8ds_gemm_mxfp4_mma refuses before anything is launched (no GPU)."""

import os

import pytest

import delayed_scaling_gemm_amd as dsg

P = 0x10000


@pytest.mark.skipif(not os.path.exists(dsg.LIB_PATH), reason="libfp8ds.so not built")
def test_refusals():
    L = dsg.lib()

    def gemm(M=64, K=128, a=P, fa=0, mma=0, lda=128):
        return L.fp8ds_gemm_mxfp4_mma(M, 64, K, a, fa, lda, P, 4, P, 128, P, 4, P, 1, 64, None, mma,
                                      None)

    for mma in (0, 1):
        assert gemm(mma=mma, fa=3) == -3 and gemm(mma=mma, K=100) == -2
        assert gemm(mma=mma, a=None) == -1 and gemm(mma=mma, a=P + 8) == -4
        assert gemm(mma=mma, lda=136) == -4 and gemm(mma=mma, M=0) == 0
    assert gemm(mma=2) == -3 and gemm(mma=-1) == -3 and gemm(mma=2, fa=2) == -3
    assert b"fp8ds_gemm_mxfp4_mma" in L.fp8ds_last_error()
