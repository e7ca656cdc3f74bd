"""Microscaled 4-bit floating point (OCP MX: e2m1 elements, 32 to a power-of-two
scale) of rows [..., d], in fp64 and by search over the sixteen values."""
from __future__ import annotations

import numpy as np

GROUP = 32
MAGNITUDE = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def quantize(x):
    """(codes uint8 [..., d/2], scale bytes uint8 [..., d/32]): the scale puts the
    group's largest magnitude into [4, 8), a code is the nearest value (ties: the
    one with mantissa bit 0), its sign the value's own."""
    x = np.asarray(x, np.float64)
    g = x.reshape(x.shape[:-1] + (-1, GROUP))
    top = np.abs(g).max(-1)
    with np.errstate(divide="ignore"):
        e = np.where(top > 0, np.floor(np.log2(top)) - 2 + 127, 0)
    e = np.clip(e, 0, 254)
    y = np.abs(g) / np.exp2(e - 127)[..., None]
    dist = np.abs(y[..., None] - MAGNITUDE)
    code = np.zeros(y.shape, np.uint8)
    best = np.full(y.shape, np.inf)
    for c in (0, 2, 4, 6, 1, 3, 5, 7):       # even codes first: they win ties
        better = dist[..., c] < best
        code[better] = c
        best = np.minimum(best, dist[..., c])
    code |= np.signbit(g).astype(np.uint8) << 3
    code = code.reshape(x.shape)
    return code[..., 0::2] | (code[..., 1::2] << 4), e.astype(np.uint8)


def dequantize(codes, scales):
    """fp64 values [..., d]."""
    codes = np.asarray(codes, np.uint8)
    c = np.stack([codes & 15, codes >> 4], -1).reshape(codes.shape[:-1] + (-1,))
    v = MAGNITUDE[c & 7] * np.where(c & 8, -1.0, 1.0)
    s = np.exp2(np.asarray(scales, np.float64) - 127)[..., None]
    return (v.reshape(v.shape[:-1] + (-1, GROUP)) * s).reshape(v.shape)
