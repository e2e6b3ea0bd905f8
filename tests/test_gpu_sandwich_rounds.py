"""The norms around a gated residual addition where a workgroup goes on to further rows, for every number
of threads a row has, and forward rows of 16385 to 32768 columns that are no multiple of 8; tolerances
as test_gpu_sandwich's."""

import pytest

torch = pytest.importorskip("torch")

import test_gpu_sandwich as base  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda"


# forward: 2048 workgroups of rows up to 8192 columns, 256 of longer ones; backward: 1024
@pytest.mark.parametrize("types", list(base.TYPES))
@pytest.mark.parametrize("R,C", [(40000, 96), (9000, 1000), (2500, 1537), (2500, 4096), (2500, 4099),
                                 (2200, 8192), (1300, 9063), (1300, 16384), (1100, 17001), (600, 24576)])
def test_every_row_as_alone(R, C, types):
    alpha = 0.5
    d = base.inputs(R, C, types, True, True)
    y = torch.empty(R, C, device=DEV)
    h, r1, r2 = base.run_forward(d, alpha, y=y)
    g = torch.Generator(device=DEV).manual_seed(R + C)
    dy = torch.randn(R, C, generator=g, device=DEV).to(d["x"].dtype)
    dres = torch.randn(R, C, generator=g, device=DEV).to(h.dtype)
    dx = torch.empty_like(dy)
    o = base.run_backward(d, h, r1, r2, dy, alpha, dres, dx=dx)
    n = 37
    for lo in (0, R // 2, R - n):
        rows = slice(lo, lo + n)
        part = {k: (v[rows] if v is not None and v.shape[0] == R else v) for k, v in d.items()}
        y2 = torch.empty(n, C, device=DEV)
        h2, s1, s2 = base.run_forward(part, alpha, y=y2)
        assert torch.equal(h2, h[rows]) and torch.equal(y2, y[rows])
        assert torch.equal(s1, r1[rows]) and torch.equal(s2, r2[rows])
        dx2 = torch.empty_like(dy[rows])
        o2 = base.run_backward(part, h2, s1, s2, dy[rows], alpha, dres[rows], dx=dx2)
        assert torch.equal(o2["dh"], o["dh"][rows]) and torch.equal(dx2, dx[rows])
        assert torch.equal(o2["drow_gate"], o["drow_gate"][rows])
    want, tol = base.backward64(dy, h, r2, d, r1, alpha, dres)
    for k in ("dgamma", "dpost_gamma", "dgate"):
        assert ((o[k].double() - want[k]).abs() <= tol[k]).all(), k


@pytest.mark.parametrize("types", list(base.TYPES))
@pytest.mark.parametrize("R,C", [(3, 16385), (2, 20001), (2, 32767), (3, 24577)])
def test_long_ragged_rows(R, C, types):
    base.test_forward(R, C, types)
    base.test_backward(R, C, types)


@pytest.mark.parametrize("types", list(base.TYPES))
@pytest.mark.parametrize("R,C", [(300, 16391), (300, 20001), (40, 32761), (300, 20000), (1100, 4099)])
def test_long_ragged_rows_in_place_are_the_others(R, C, types):
    base.test_ragged_rows_in_place_are_the_others(R, C, types)
