"""Transposed copies whose tiles no grid can count are refused (no GPU: addresses are never
dereferenced)."""

import os

import pytest

import delayed_scaling_gemm_amd as dsg

P = 0x10000


@pytest.mark.skipif(not os.path.exists(dsg.LIB_PATH), reason="libfp8ds.so not built")
@pytest.mark.parametrize("cols", [1 << 31, 1 << 33])
def test_columns_past_the_grid(cols):
    L = dsg.lib()
    assert L.fp8ds_cast(P, 1, 1, cols, 0, P, P, P, None, None, None, None) == -2
    assert L.fp8ds_cast_acc(P, 1, 1, cols, 0, P, P, P, None, None, None, None) == -2
    assert L.fp8ds_cast_current(P, 1, 1, cols, 0, 0, P, P, P, None, P, None, None) == -2
    assert L.fp8ds_adamw(P, P, 1, P, P, 1, cols, 1e-3, 0.9, 0.999, 1e-8, 0.0, 1.0, 1, None, 0, P, P, P,
                         None, None, None, None) == -2
