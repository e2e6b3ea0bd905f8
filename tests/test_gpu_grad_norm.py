"""GPU parity of the gradient norm, the clip and the clipped AdamW step.

The norm's sums are fp64 and it is rounded once: at most 2^-24 relative, and the fp64
sum of n squares adds n 2^-53; coef likewise.  The clip is one fp32 product and one
rounding: bit for bit from the coefficient that the GPU has."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import delayed_scaling_gemm_amd as dsg  # noqa: E402
from oracle import norm as onorm  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0**-24


def tensors(sizes, types, seed, mag=1e-3):
    g = torch.Generator().manual_seed(seed)
    return [(torch.randn(n, generator=g) * mag * (1 + i)).to(t).to(DEV)
            for i, (n, t) in enumerate(zip(sizes, types))]


def norm_of(grads, max_norm=1.0, grad_scale=1.0):
    work = torch.full((dsg.fp8ds_grad_norm_workspace(),), 0xFF, dtype=torch.uint8, device=DEV)
    norm, coef = torch.empty(1, device=DEV), torch.empty(1, device=DEV)
    dsg.fp8ds_grad_norm(grads, max_norm, norm, coef, work, grad_scale=grad_scale)
    torch.cuda.synchronize()
    return norm, coef


def check(grads, max_norm=1.0, grad_scale=1.0):
    norm, coef = norm_of(grads, max_norm, grad_scale)
    n, c = onorm.grad_norm([g.float().cpu().numpy() for g in grads], grad_scale, max_norm)
    assert abs(float(norm) - n) <= 2 * U * n
    assert abs(float(coef) - c) <= 2 * U * c
    return norm, coef


BF, F32 = torch.bfloat16, torch.float32
SETS = [([1], [BF]), ([0, 5, 0], [BF, F32, F32]), ([8192, 8193, 8191, 1], [BF, F32, BF, F32]),
        ([65536], [BF]), ([65537], [F32]), ([300000, 7, 100001], [BF, BF, F32]),
        ([3] * 500, [BF, F32] * 250), ([5000] * 300, [F32, BF] * 150), ([40_000_001], [BF])]


@pytest.mark.parametrize("sizes,types", SETS)
def test_norm(sizes, types):
    grads = tensors(sizes, types, len(sizes))
    check(grads, 0.5)
    check(grads, 1e9, 0.25)
    a, b = norm_of(grads), norm_of(grads)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_norm_of_nothing_and_of_zeros():
    assert float(norm_of([])[0]) == 0.0
    n, c = norm_of([torch.zeros(10, device=DEV)])
    assert float(n) == 0.0 and float(c) == 1.0


def test_norm_range_and_non_finite():
    for v in (1e30, 1e-30):  # squares beyond fp32
        g = torch.full((1000,), v, device=DEV)
        n, _ = norm_of([g])
        assert abs(float(n) / (float(g[0]) * np.sqrt(1000)) - 1) < 4 * U
    g = torch.ones(70000, device=DEV)
    g[3] = float("inf")
    n, c = norm_of([g])
    assert np.isinf(float(n)) and float(c) == 0.0
    g[4] = float("nan")
    n, c = norm_of([g])
    assert np.isnan(float(n)) and np.isnan(float(c))


def test_norm_of_unaligned_slices():
    base = tensors([20001], [BF], 3)[0]
    check([base[1:], base[3:20000], tensors([999], [F32], 4)[0][1:]])


@pytest.mark.parametrize("it", [BF, F32])
@pytest.mark.parametrize("ot", [BF, F32])
def test_clip_into_other_tensors(it, ot):
    sizes = [1, 0, 4, 1023, 8192, 8197, 100003] + [3] * 150
    grads = tensors(sizes, [it] * len(sizes), 5)
    out = [torch.full((n,), 7.0, dtype=ot, device=DEV) for n in sizes]
    _, coef = norm_of(grads, 0.01)
    assert float(coef) < 1.0
    dsg.fp8ds_grad_clip(grads, coef, out)
    torch.cuda.synchronize()
    for g, o in zip(grads, out):
        assert torch.equal(o, (g.float() * coef).to(ot))


def test_clip_in_place_slices_and_unit_coefficient():
    base = tensors([5001], [BF], 6)[0]
    whole, grads = base.clone(), [base[1:2000], base[2001:5000]]
    ref = [g.clone() for g in grads]
    one = torch.ones(1, device=DEV)
    dsg.fp8ds_grad_clip(grads, one)
    torch.cuda.synchronize()
    assert torch.equal(base, whole)
    half = torch.full((1,), 0.3, device=DEV)
    dsg.fp8ds_grad_clip(grads, half)
    torch.cuda.synchronize()
    for g, r in zip(grads, ref):
        assert torch.equal(g, (r.float() * half).to(BF))
    assert torch.equal(base[[0, 2000, 5000]], whole[[0, 2000, 5000]])
    out = [torch.zeros_like(r) for r in ref]
    dsg.fp8ds_grad_clip(ref, one, out)  # another tensor is written whatever the coefficient
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, ref))


def test_adamw_reads_the_coefficient():
    """fp8ds_adamw_clip equals fp8ds_adamw given fl32(grad_scale * coef) from the host, and
    a norm that is not finite skips the step."""
    for shape in ((64, 96), (128, 256), (1000,)):
        w0 = torch.randn(shape, device=DEV)
        g = (torch.randn(shape, device=DEV) * 3).to(BF)
        norm, coef = norm_of([g.view(-1)], 0.7, 0.5)
        sc = torch.full((1,), 50.0, device=DEV)
        res = []
        for use in (True, False):
            w, m, v = w0.clone(), torch.zeros_like(w0), torch.zeros_like(w0)
            q = torch.empty(shape, dtype=torch.uint8, device=DEV)
            qt = torch.empty(w0.numel(), dtype=torch.uint8, device=DEV) if len(shape) == 2 else None
            scale = np.float32(0.5) * np.float32(coef.item())
            dsg.fp8ds_adamw(w, g, m, v, 1e-2, 0.9, 0.99, 1e-8, 0.1, 1,
                            grad_scale=0.5 if use else float(scale), grad_amax=norm, scale=sc, q=q,
                            q_t=qt, grad_coef=coef if use else None)
            torch.cuda.synchronize()
            res.append([w, m, v, q] + ([qt] if qt is not None else []))
        assert all(torch.equal(a, b) for a, b in zip(*res))
        w, m, v = w0.clone(), torch.zeros_like(w0), torch.zeros_like(w0)
        bad = torch.full((1,), float("inf"), device=DEV)
        dsg.fp8ds_adamw(w, g, m, v, 1e-2, 0.9, 0.99, 1e-8, 0.1, 1, grad_amax=bad,
                        grad_coef=torch.zeros(1, device=DEV))
        torch.cuda.synchronize()
        assert torch.equal(w, w0) and not m.any()


def test_graph_replays():
    grads = tensors([100000, 17, 4096], [BF, F32, F32], 9)
    out = [torch.empty_like(g) for g in grads]
    work = torch.empty(dsg.fp8ds_grad_norm_workspace(), dtype=torch.uint8, device=DEV)
    norm, coef = torch.empty(1, device=DEV), torch.empty(1, device=DEV)

    def both():
        dsg.fp8ds_grad_norm(grads, 0.1, norm, coef, work)
        dsg.fp8ds_grad_clip(grads, coef, out)

    both()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    for k in range(3):
        for g in grads:
            g.copy_(torch.randn(g.shape, device=DEV) * (k + 1))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out + [norm, coef]]
        both()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, out + [norm, coef]))
