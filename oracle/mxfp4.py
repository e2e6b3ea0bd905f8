"""MXFP4: E2M1 elements in blocks of 32 that share an E8M0 scale (oracle; test
infrastructure only).

OCP Microscaling Formats (MX) specification v1.0: E2M1 has a sign, two exponent bits
(bias 1) and one mantissa bit; codes 0..7 are 0, 0.5, 1, 1.5, 2, 3, 4, 6, code | 8 the
negatives; no infinity, no NaN; ``emax`` 2.  A block's scale is
``2**(floor(log2(amax)) - 2)``, its elements the nearest E2M1 values of ``v / scale`` (ties
to the even code, saturating at 6).  Readings as for MXFP8: the exponent is clamped to
[-127, 127], a zero block takes code 0, a block with a NaN or an infinity takes code
255 (its elements, which have no NaN, are stored as 6).  Element 2 i of a row is the low
half of byte i.
"""

from __future__ import annotations

import numpy as np

from .mx import BLOCK, E8M0_BIAS, E8M0_NAN

VALUES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
EMAX = 2
NAN_BLOCK_CODE = 7


def decode(codes) -> np.ndarray:
    """Values of 4-bit codes (fp64)."""
    c = np.asarray(codes, dtype=np.int64)
    return np.where(c & 8, -1.0, 1.0) * VALUES[c & 7]


def encode(v) -> np.ndarray:
    """Nearest code of each (finite) value by search over the eight magnitudes: the
    smaller distance wins, of two equal ones the even code."""
    v = np.asarray(v, dtype=np.float64)
    a = np.abs(v)
    best = np.zeros(a.shape, dtype=np.int64)
    dist = np.abs(a - VALUES[0])
    for c in range(1, 8):
        d = np.abs(a - VALUES[c])
        take = (d < dist) | ((d == dist) & (c % 2 == 0))
        best, dist = np.where(take, c, best), np.where(take, d, dist)
    return (best | np.where(np.signbit(v), 8, 0)).astype(np.uint8)


def pack(codes: np.ndarray) -> np.ndarray:
    return (codes[..., 0::2] | (codes[..., 1::2] << 4)).astype(np.uint8)


def unpack(q: np.ndarray) -> np.ndarray:
    q = np.asarray(q, dtype=np.uint8)
    return np.stack([q & 15, q >> 4], axis=-1).reshape(*q.shape[:-1], 2 * q.shape[-1])


def scale_value(codes) -> np.ndarray:
    c = np.asarray(codes, dtype=np.int64)
    return np.where(c == E8M0_NAN, np.nan, np.ldexp(1.0, np.where(c == E8M0_NAN, 0, c - E8M0_BIAS)))


def cast(x: np.ndarray):
    """(packed codes [R, C / 2], E8M0 codes [R, C / 32]) of a 2-D fp32 array."""
    x = np.asarray(x, dtype=np.float32).astype(np.float64)
    R, C = x.shape
    b = x.reshape(R, C // BLOCK, BLOCK)
    bad = ~np.isfinite(b).all(axis=-1)
    b = np.where(bad[..., None], 0.0, b)
    amax = np.abs(b).max(axis=-1)
    _, e = np.frexp(amax)
    E = np.clip(e.astype(np.int64) - 1 - EMAX, -E8M0_BIAS, E8M0_BIAS)
    sc = np.where(bad, E8M0_NAN, np.where(amax == 0, 0, E + E8M0_BIAS))
    codes = encode(b / np.ldexp(1.0, np.where(bad, 0, sc - E8M0_BIAS))[..., None])
    codes = np.where(bad[..., None], NAN_BLOCK_CODE, codes).reshape(R, C).astype(np.uint8)
    return pack(codes), sc.astype(np.uint8)


def dequant(q: np.ndarray, scales: np.ndarray) -> np.ndarray:
    """Values in fp64."""
    return decode(unpack(q)) * np.repeat(scale_value(scales), BLOCK, axis=-1)
