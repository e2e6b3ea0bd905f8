"""fp8ds_cast_rowwise with more rows than one grid of a workgroup each takes."""

import pytest

torch = pytest.importorskip("torch")

import delayed_scaling_gemm_amd as dsg  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("cols", [3, 8])
def test_rows_past_one_grid(dtype, cols):
    rows = (1 << 24) + 33  # of 256 threads: 2^32 and more
    g = torch.Generator(device=DEV).manual_seed(cols)
    x = torch.randn(rows, cols, generator=g, device=DEV).to(dtype)
    q = torch.full((rows, cols), 9, dtype=torch.uint8, device=DEV)
    s, inv, am = (torch.full((rows,), 9.0, device=DEV) for _ in range(3))
    dsg.fp8ds_cast_rowwise(x, dsg.E4M3, 0, q, s, inv, am)
    torch.cuda.synchronize()
    a = x.float().abs().amax(1)
    assert torch.equal(am, a)
    # (quotients of fp32 numbers taken in fp64 round to the fp32 quotients)
    want = torch.where(a > 0, (448.0 / a.double()).float(), torch.ones_like(a))
    assert torch.equal(s, want) and torch.equal(inv, (1.0 / s.double()).float())
    v = (x.float() * s[:, None]).clamp(-448, 448)
    assert torch.equal(q, v.to(torch.float8_e4m3fn).view(torch.uint8))
