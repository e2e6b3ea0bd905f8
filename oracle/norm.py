"""RMSNorm with the residual's addition, its backward pass, and the global gradient
norm (oracle; test infrastructure only), in fp64 from the definitions:

    h = x + residual (rounded to the residual's type)
    r = 1 / sqrt(mean(h**2) + eps),   y = h r gamma
    dx = r (g - xhat mean(g xhat)) + dres,  dgamma = sum_rows dy xhat
    with xhat = h r, g = dy gamma
    norm = grad_scale sqrt(sum g**2),  coef = min(1, max_norm / (norm + 1e-6))
"""

from __future__ import annotations

import numpy as np

from . import bf16


def to_bf16(x):
    """fp64 values of x rounded to BF16."""
    return bf16.widen(bf16.round_to_bf16_vec(np.asarray(x, np.float64))).astype(np.float64)


def residual_sum(x, res, h_bf16: bool):
    """h as stored: the fp32 sum, rounded once more where the stream is BF16."""
    h = np.asarray(x, np.float64)
    if res is None:
        return h
    h = (h + np.asarray(res, np.float64)).astype(np.float32).astype(np.float64)
    return to_bf16(h).reshape(h.shape) if h_bf16 else h


def forward(h, gamma, eps: float):
    """(r [rows], y [rows, cols]) in fp64."""
    h = np.asarray(h, np.float64)
    with np.errstate(divide="ignore", invalid="ignore", over="ignore"):
        r = 1.0 / np.sqrt((h * h).sum(axis=1) / h.shape[1] + float(np.float32(eps)))
        return r, h * r[:, None] * np.asarray(gamma, np.float64)


def backward(dy, h, r, gamma, dres=None):
    """(dx, dgamma, bound terms): the last is what the fp32 error of dx is a multiple of."""
    dy, h, r, gamma = (np.asarray(a, np.float64) for a in (dy, h, r, gamma))
    xhat = h * r[:, None]
    g = dy * gamma
    mean = (g * xhat).sum(axis=1, keepdims=True) / h.shape[1]
    dx = r[:, None] * (g - xhat * mean)
    terms = np.abs(r[:, None]) * (np.abs(g) + np.abs(xhat) *
                                  np.abs(g * xhat).sum(axis=1, keepdims=True) / h.shape[1])
    if dres is not None:
        dx = dx + np.asarray(dres, np.float64)
        terms = terms + np.abs(dres)
    return dx, (dy * xhat).sum(axis=0), terms


def grad_norm(grads, grad_scale: float, max_norm: float):
    total = sum(float((np.asarray(g, np.float64) ** 2).sum()) for g in grads)
    norm = grad_scale * np.sqrt(total)
    return norm, min(1.0, max_norm / (norm + 1e-6))
