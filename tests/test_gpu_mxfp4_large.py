"""The plain MXFP4 cast of large tensors (8 pieces a thread, from 8 x 256 pieces of 16 bytes per CU
on), bit for bit with the oracle, and back; MXFP4Linear serving few tokens."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import delayed_scaling_gemm_amd as dsg  # noqa: E402
from delayed_scaling_gemm_amd.linear import MXFP4Linear  # noqa: E402
from oracle import mxfp4 as o4  # noqa: E402
from tests.parity import bf16_ulp  # noqa: E402
from tests.test_gpu_mxfp4 import bound, values  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("bf16,shape", [(True, (1025, 4128)), (True, (131073, 32)), (False, (701, 3008)),
                                        (False, (3, 1048608))])
def test_cast_and_values(shape, bf16):
    rows, cols = shape
    cus = torch.cuda.get_device_properties(0).multi_processor_count
    pieces = rows * cols // (8 if bf16 else 4)
    assert pieces >= 8 * 256 * cus and pieces % 2048  # a last workgroup that is not full
    x, ref = values(rows, cols, rows + cols, bf16)
    q = torch.full((rows * cols // 2 + 64,), 9, dtype=torch.uint8, device=DEV)
    s = torch.full((rows * cols // 32 + 64,), 9, dtype=torch.uint8, device=DEV)
    dsg.fp8ds_cast_mxfp4(x, q, s)
    y = torch.empty(rows, cols, dtype=torch.bfloat16, device=DEV)
    dsg.fp8ds_dequant_mxfp4(q, s, y)
    torch.cuda.synchronize()
    oq, os_ = o4.cast(ref)
    np.testing.assert_array_equal(s[:-64].cpu().numpy().reshape(os_.shape), os_)
    np.testing.assert_array_equal(q[:-64].cpu().numpy().reshape(oq.shape), oq)
    assert bool((q[-64:] == 9).all()) and bool((s[-64:] == 9).all())
    np.testing.assert_array_equal(y.float().cpu().numpy().astype(np.float64), o4.dequant(oq, os_))


@pytest.mark.parametrize("K,N", [(416, 160), (4096, 96), (96, 9024)])
def test_forward_of_few_tokens(K, N):
    rng = np.random.default_rng(K)
    x = torch.from_numpy(rng.standard_normal((288, K))).to(DEV).to(torch.bfloat16)
    w = torch.from_numpy(0.02 * rng.standard_normal((K, N))).to(DEV).to(torch.bfloat16)
    layer = MXFP4Linear(device=DEV)
    layer.quantize(w)
    wv = o4.dequant(*o4.cast(np.ascontiguousarray(w.float().cpu().numpy().T)))
    for m in (1, 7, 16, 17, 288):
        y = layer.forward(x[:m])
        torch.cuda.synchronize()
        xv = o4.dequant(*o4.cast(x[:m].float().cpu().numpy()))
        acc, bd = xv @ wv.T, bound(xv, wv, K, dsg.E2M1)
        got = y.float().cpu().numpy()
        assert got.shape == (m, N)
        assert (np.abs(got - acc) <= bd + bf16_ulp(np.abs(acc) + bd) / 2).all(), m
