"""The gradient norm and the clip over more elements than one launch of the clip takes (2^33)."""

import pytest

torch = pytest.importorskip("torch")

import delayed_scaling_gemm_amd as dsg  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda"


def test_clip_of_more_than_one_launch():
    # a first tensor that ends inside a chunk, then one that spans the launches, then others
    sizes = [5001, (1 << 33) + 12345, 0, 70000, 3]
    bf = torch.bfloat16
    grads = [torch.ones(n, dtype=bf, device=DEV) for n in sizes]
    big = grads[1]
    big[::4099] = 3.0
    big[-5:] = -2.0
    grads[3][7] = 5.0
    squares = sum(float(n) for n in sizes)
    n3 = len(range(0, sizes[1], 4099))
    in_tail = [i for i in range(sizes[1] - 5, sizes[1]) if i % 4099 == 0]
    squares += 8.0 * (n3 - len(in_tail)) + 5 * 3.0 + 24.0
    norm, coef = torch.empty(1, device=DEV), torch.empty(1, device=DEV)
    ws = torch.empty(dsg.fp8ds_grad_norm_workspace(), dtype=torch.uint8, device=DEV)
    dsg.fp8ds_grad_norm(grads, 1.0, norm, coef, ws)
    torch.cuda.synchronize()
    assert abs(float(norm) - squares**0.5) <= 2 * 2.0**-24 * squares**0.5  # exact sum, two roundings
    half = torch.full((1,), 0.5, device=DEV)
    dsg.fp8ds_grad_clip(grads, half)
    torch.cuda.synchronize()
    step = 1 << 30
    for i in range(0, sizes[1], step):
        part = big[i:i + step]
        want = torch.full((part.numel(),), 0.5, dtype=bf, device=DEV)
        want[(-i) % 4099::4099] = 1.5
        if i + step >= sizes[1]:
            want[-5:] = -1.0
        assert torch.equal(part, want), i
    assert bool((grads[0] == 0.5).all()) and bool((grads[4] == 0.5).all())
    assert float(grads[3][7]) == 2.5 and int((grads[3] == 0.5).sum()) == sizes[3] - 1
