"""The gradient norm where a workgroup's chunks (8192 elements each) span several tensors: more
than 1024 chunks a launch; and AdamW of a Linear that reads the coefficient and the norm."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import delayed_scaling_gemm_amd as dsg  # noqa: E402
from delayed_scaling_gemm_amd.linear import DelayedScalingLinear  # noqa: E402
from tests.test_gpu_grad_norm import check, norm_of, tensors  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32


def chunks(sizes):
    return sum(-(-n // 8192) for n in sizes)


@pytest.mark.parametrize("sizes", [
    [9_000_001, 0, 5, 8193, 3_000_000, 70_001],
    [85_000 + i for i in range(128)],                      # 11 chunks each, two a workgroup
    [0, 0] + [90_001] * 100 + [0] * 60 + [8191] * 200,     # three launches
    [1] * 127 + [40_000_000]])                             # many tensors in the first workgroups
def test_norm(sizes):
    assert max(chunks([n for n in sizes if n][i:i + 128]) for i in range(0, len(sizes), 128)) > 1024
    types = [BF if i % 3 else F32 for i in range(len(sizes))]
    grads = tensors(sizes, types, len(sizes))
    check(grads, 0.5)
    a, b = norm_of(grads), norm_of(grads)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    # each tensor is counted once and whole: its last element alone
    for i in {0, len(sizes) // 2, len(sizes) - 1}:
        if sizes[i]:
            zeros = [torch.zeros_like(g) for g in grads]
            zeros[i][-1] = 3.0
            assert float(norm_of(zeros)[0]) == 3.0


def test_adamw_step_of_a_linear_reads_the_coefficient_and_the_norm():
    M, K, N = 64, 128, 96
    g = torch.Generator(device=DEV).manual_seed(0)
    x, dy = (torch.randn(s, generator=g, device=DEV).to(BF) for s in ((M, K), (M, N)))
    w0 = torch.randn(K, N, generator=g, device=DEV)

    def run(coef, norm, plain):
        lin = DelayedScalingLinear(device=DEV)
        w, m, v = w0.clone(), torch.zeros_like(w0), torch.zeros_like(w0)
        lin.step(x, w, dy)
        dw = lin._bufs["dw"].clone()
        if plain:  # the same update from the separate call, its factor from the host
            wq, wqt = torch.empty(K, N, dtype=torch.uint8, device=DEV), torch.empty(N, K, dtype=torch.uint8, device=DEV)
            dsg.fp8ds_adamw(w, dw, m, v, 1e-2, 0.9, 0.999, 1e-8, 0.1, 1,
                            grad_scale=float(np.float32(0.5) * np.float32(coef.item())),
                            scale=lin.scale[1:2], q=wq, q_t=wqt)
        else:
            lin.adamw_step(w, m, v, 1e-2, 1, weight_decay=0.1, grad_scale=0.5, grad_coef=coef,
                           grad_norm=norm)
            wq, wqt = lin._bufs["wq"], lin._bufs["wqt"]
        torch.cuda.synchronize()
        return [w, m, v, wq, wqt], dw

    _, dw = run(torch.ones(1, device=DEV), None, True)
    norm, coef = norm_of([dw], 0.3, 0.5)
    assert 0 < float(coef) < 1
    for n in (norm, None):
        got, want = run(coef, n, False)[0], run(coef, None, True)[0]
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    # another tensor's infinity, seen in the norm, skips this layer too
    got = run(torch.zeros(1, device=DEV), torch.full((1,), float("inf"), device=DEV), False)[0]
    assert torch.equal(got[0], w0) and not got[1].any() and not got[2].any()
