"""Muon's direction where the norm or eps is near the ends of fp32's range.

X = U / (|U|_F + eps) is one fp32 rounding of a quotient in 64 bits: X may be off by 2^-24 of each
element whatever the norm is.  Gradients that differ by a power of two, without a momentum and with
an eps that is lost beside the norm, have X of the same bits."""

import pytest

torch = pytest.importorskip("torch")

import delayed_scaling_gemm_amd as dsg  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda"
R, C = 50, 90


def direction(g, eps):
    o = torch.empty(R, C, device=DEV)
    ws = torch.full((dsg.fp8ds_muon_workspace(R, C),), 0xFF, dtype=torch.uint8, device=DEV)
    dsg.fp8ds_muon_direction(g, o, ws, eps=eps)
    return o


def gauss():
    return torch.randn(R, C, generator=torch.Generator(device=DEV).manual_seed(3), device=DEV)


@pytest.mark.parametrize("eps", [1e-7, 1e-37, 2e-39, 1e-42, 2.0 ** -149])
def test_zero_update_gives_zero(eps):
    assert (direction(torch.zeros(R, C, device=DEV), eps) == 0).all()


@pytest.mark.parametrize("eps", [1e-40, 2.0 ** -149])
def test_tiny_update_and_tiny_eps(eps):
    """|U| of about 2^-126 with elements down to 2^-140 and an eps below the normal numbers."""
    whole = torch.round(gauss() * 64)
    g = whole * 2.0 ** -138  # exact in fp32's subnormal numbers too
    assert torch.isfinite(direction(g, eps)).all()
    if eps == 2.0 ** -149:  # 2^-23 of the norm and less
        e = direction(whole, 1e-30).double()
        # each singular value of X moves by at most 2^-23 of itself, which five steps multiply by at
        # most 3.4445^5 = 485; either side is off the iteration in 64 bits by at most 7e-5
        assert (direction(g, eps).double() - e).norm() <= 485 * 2.0 ** -23 + 2 * 7e-5 * e.norm()


@pytest.mark.parametrize("power", [60, 118, 122, 124])
def test_large_norms(power):
    """Norms up to 2^130: above 2^126 the reciprocal is no normal number of fp32."""
    g = gauss().clamp_(-7, 7)
    assert torch.equal(direction(g * 2.0 ** power, 1e-7), direction(g, 1e-30))


@pytest.mark.parametrize("eps,size", [(1e-7, 1e-8), (1e-7, 1e-12), (1e-7, 1e-20), (1e-7, 1e-28), (1.0, 1e-3),
                                      (1.0, 1e-9), (1e20, 1e-5)])
@pytest.mark.parametrize("rows,cols", [(50, 90), (64, 900), (2000, 300)])
@pytest.mark.parametrize("steps", [5, 8])
def test_updates_far_below_eps(rows, cols, steps, eps, size):
    """X is then far below 1 and grows by 3.4445 a step at most: the contract's 1e-5 of the result."""
    g = size * torch.randn(rows, cols, generator=torch.Generator(device=DEV).manual_seed(4), device=DEV)
    o = torch.empty(rows, cols, device=DEV)
    ws = torch.full((dsg.fp8ds_muon_workspace(rows, cols),), 0xFF, dtype=torch.uint8, device=DEV)
    dsg.fp8ds_muon_direction(g, o, ws, eps=eps, steps=steps)
    x = g.double() / (g.double().norm() + torch.tensor(eps, dtype=torch.float32).double())
    x = x.t().contiguous() if rows > cols else x
    for _ in range(steps):
        A = x @ x.t()
        x = 3.4445 * x + (-4.7750 * A + 2.0315 * (A @ A)) @ x
    x = x.t() if rows > cols else x
    assert (o.double() - x).norm() <= 1e-5 * x.norm()
