"""Pins of the oracles of RMSNorm, the gradient norm and MXFP4 (CPU)."""

import numpy as np
import pytest

from oracle import mxfp4 as o4
from oracle import norm as onorm


def test_e2m1_codes_and_ties():
    assert o4.decode(np.arange(8)).tolist() == [0, 0.5, 1, 1.5, 2, 3, 4, 6]
    assert (o4.encode(o4.decode(np.arange(16))) == np.arange(16)).all()
    # ties go to the even code: 0.25 -> 0, 0.75 -> 1, 1.25 -> 1, 1.75 -> 2, 2.5 -> 2, 3.5 -> 4, 5 -> 4
    v = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.0, 100.0])
    assert o4.decode(o4.encode(v)).tolist() == [0, 1, 1, 2, 2, 4, 4, 6, 6]
    assert (o4.encode(-v) == (o4.encode(v) | 8)).all()


def test_mxfp4_worked_block():
    x = np.zeros((1, 32), np.float32)
    x[0, :4] = [7.0, -1.0, 0.3, 5.0]       # amax 7: floor(log2) = 2, scale 2^0
    q, s = o4.cast(x)
    assert s[0, 0] == 127
    assert o4.dequant(q, s)[0, :4].tolist() == [6.0, -1.0, 0.5, 4.0]
    assert q[0, 0] == (7 | ((2 | 8) << 4))


def test_mxfp4_degenerate_blocks():
    x = np.ones((1, 128), np.float32)
    x[0, :32] = 0.0
    x[0, 40] = np.inf
    x[0, 70] = np.nan
    x[0, 96:] = np.float32(2.0**-140)
    q, s = o4.cast(x)
    assert s[0].tolist() == [0, 255, 255, 0]
    d = o4.dequant(q, s)
    assert (d[0, :32] == 0).all() and np.isnan(d[0, 32:96]).all() and (d[0, 96:] == 0).all()


def test_norm_closed_forms():
    # a constant row has r = 1 / sqrt(c^2 + eps), y = sign(c) gamma for eps = 0
    h = np.full((2, 10), -3.0)
    r, y = onorm.forward(h, np.arange(10.0), 0.0)
    assert np.allclose(r, 1 / 3) and np.allclose(y, -np.arange(10.0))
    # y does not depend on the row's magnitude
    rng = np.random.default_rng(0)
    h = rng.standard_normal((3, 50))
    assert np.allclose(onorm.forward(h, np.ones(50), 0.0)[1], onorm.forward(8 * h, np.ones(50), 0.0)[1])


@pytest.mark.parametrize("with_res", [False, True])
def test_norm_backward_against_differences(with_res):
    rng = np.random.default_rng(1)
    rows, cols, eps = 3, 17, 1e-3
    h, dy = rng.standard_normal((rows, cols)), rng.standard_normal((rows, cols))
    gamma, dres = rng.standard_normal(cols), rng.standard_normal((rows, cols))

    def loss(h, gamma):
        return (onorm.forward(h, gamma, eps)[1] * dy).sum() + ((h * dres).sum() if with_res else 0.0)

    r = onorm.forward(h, gamma, eps)[0]
    dx, dg, _ = onorm.backward(dy, h, r, gamma, dres if with_res else None)
    step = 1e-6
    for i in range(rows):
        for j in range(cols):
            e = np.zeros_like(h)
            e[i, j] = step
            d = (loss(h + e, gamma) - loss(h - e, gamma)) / (2 * step)
            assert abs(d - dx[i, j]) < 1e-7 * max(1, abs(d))
    for j in range(cols):
        e = np.zeros(cols)
        e[j] = step
        assert abs((loss(h, gamma + e) - loss(h, gamma - e)) / (2 * step) - dg[j]) < 1e-7


def test_grad_norm_worked():
    n, c = onorm.grad_norm([np.array([3.0]), np.array([4.0, 0.0])], 1.0, 1.0)
    assert n == 5.0 and c == 1.0 / (5.0 + 1e-6)
    assert onorm.grad_norm([np.array([0.3])], 0.5, 1.0) == (0.15, 1.0)
