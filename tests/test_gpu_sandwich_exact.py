"""h of the norms around a residual addition is its exact value, rounded to fp32 and then to the stream's
type (rows of up to 16384 columns).

r1, k and the addition are in 64 bits; what remains are the squares, added in pairs in fp32.  A pair is off
by at most 2^-24 of itself (BF16 squares are exact; FP32 ones add 2^-24), so r1 by at most half of
that: 2^-25, with FP32 x 2^-24.  So much of |p|, and half a unit, is what an FP32 h may be off by.  (An
average over the pairs, 2^-28, was wrong as a bound of 30000 rows of 96 columns.)
A BF16 h may lie on the other side of a border only if the fp32 sum differs and lies next to a border,
which 3 in 65536 do.  It differs for err / 2^-24 of elements with err the error of p over |h|: the pairs'
errors are uniform, 2^-25.8, and of either sign; a ninth of the pairs carries half of the sum here, so
11 of them at C = 96 leave 2^-25.8 / sqrt(11) / 2 = 2^-28.5 of p, half of it for |p| <= |h|: 1e-6 of the elements,
less for more columns.  Asked for is 3e-6; the expression in fp32 gives 2e-5.  Where the sum cancels nothing is
asked."""

import pytest

torch = pytest.importorskip("torch")

import test_gpu_sandwich as base  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("types", list(base.TYPES))
@pytest.mark.parametrize("R,C", [(30000, 96), (3000, 1000), (3000, 1537), (2000, 4096), (1200, 4099), (1000, 8192),
                                 (700, 9063), (600, 16384)])
@pytest.mark.parametrize("gates", [False, True])
def test_h_is_rounded_once(R, C, types, gates):
    d = base.inputs(R, C, types, gates, gates, seed=6)
    d["res"] = d["res"].float().mul(0.5).to(d["res"].dtype)
    h, r1, _ = base.run_forward(d, 0.7)
    alpha = float(torch.tensor(0.7, dtype=torch.float32))
    e1, p, exact = base.forward64(d, alpha)
    eps = float(torch.tensor(base.EPS1, dtype=torch.float32))
    x = d["x"].double()
    e1b = 1 / torch.sqrt((x * x).mean(1) + eps)  # eps and alpha are fp32 arguments
    p = p * (e1b / e1)[:, None]
    exact = d["res"].double() + p
    err = 2.0 ** (-24 if d["x"].dtype == torch.float32 else -25)
    assert ((r1.double() - e1b).abs() <= (base.U + err) * e1b).all()
    if h.dtype == torch.float32:
        assert ((h.double() - exact).abs() <= base.U * exact.abs() + err * p.abs() + 1e-38).all()
    else:
        other = (h != exact.float().to(h.dtype)) & (exact.abs() >= p.abs())
        assert int(other.sum()) <= 3e-6 * R * C
