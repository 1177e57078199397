"""Storage in 8 bits and the layer on it, in numpy and 64 bits (the oracle of the
8-bit calls)."""
from __future__ import annotations

import numpy as np


def quantize_rows(x, block: int = 0):
    """codes int8 and scales fp32 of the rows of x, or of runs of `block` columns.

    a = max |x|, scale = fp32(a / 127), code = nearest integer to 127 x / a (ties
    to the even one); zero rows: scale 0; rows with a NaN or infinity: scale NaN,
    codes 0."""
    x = np.asarray(x, np.float64)
    v = x.reshape(x.shape[0], -1, block) if block else x[:, None, :]
    a = np.abs(v).max(-1)
    bad = ~np.isfinite(v).all(-1)
    a = np.where(bad, 0.0, a)
    safe = np.where(a == 0, 1.0, a)
    n = np.where((a == 0)[..., None], 0.0, 127.0 * np.where(bad[..., None], 0.0, v) / safe[..., None])
    codes = np.rint(n).astype(np.int8).reshape(x.shape)
    scale = a.astype(np.float32) / np.float32(127.0)
    scale = np.where(bad, np.float32(np.nan), scale)
    return codes, (scale if block else scale[:, 0])


def values(codes, scale):
    """What codes and scales stand for, in 64 bits."""
    c, s = np.asarray(codes, np.float64), np.asarray(scale, np.float64)
    if s.ndim == 1:
        return c * s[:, None]
    return (c.reshape(*s.shape, -1) * s[..., None]).reshape(c.shape)


def silu(g):
    g = np.asarray(g, np.float64)
    return g / (1.0 + np.exp(-g))


def silu_mul_grad(dH, g, u):
    """(dG, dU) of H = silu(g) u."""
    sig = 1.0 / (1.0 + np.exp(-np.asarray(g, np.float64)))
    return dH * u * sig * (1.0 + g * (1.0 - sig)), dH * g * sig
