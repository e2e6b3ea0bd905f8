"""The transposing MXFP4 cast refuses a grid that no launch can have (no GPU: addresses are never
dereferenced)."""

import os

import pytest

import delayed_scaling_gemm_amd as dsg

P = 0x10000


@pytest.mark.skipif(not os.path.exists(dsg.LIB_PATH), reason="libfp8ds.so not built")
@pytest.mark.parametrize("cols", [1 << 31, (1 << 31) + 32, 1 << 33])
def test_columns_past_the_grid(cols):
    L = dsg.lib()
    assert L.fp8ds_cast_mxfp4(P, 1, 32, cols, P, P, P, P, None) == -2
    assert b"tiles" in L.fp8ds_last_error()
