"""Linear layers in 8-bit integers in fp64: symmetric codes with a scale per
row, and the product of codes.

A code is the exact quotient x / s rounded to the nearest integer, halves to
even.  fp64 division decides every case: x has 11 significant bits at most and
s 24, so a quotient that is not half a step differs from it by 2^-34 of itself
or more.
"""

from __future__ import annotations

import numpy as np

from . import linear as ol

__all__ = ["quantize", "linear"]


def quantize(x):
    """``(codes, scales)`` of the rows of x (values of 16-bit types)."""
    x = np.asarray(x, dtype=np.float64)
    finite = np.isfinite(x).all(axis=1)
    most = np.where(finite, np.abs(np.where(np.isfinite(x), x, 0.0)).max(axis=1, initial=0.0), np.nan)
    s = (most / 127.0).astype(np.float32)
    live = finite & (s > 0)
    by = np.where(live, s, 1.0).astype(np.float64)
    q = np.rint(np.where(live[:, None], np.where(np.isfinite(x), x, 0.0) / by[:, None], 0.0))
    return q.astype(np.int8), s


def linear(xq, sx, wq, sw, bias=None, name="none", residual=None):
    """``(y, z)``: z = sx sw (xq Wq^T) + bias, y = act(z) + residual."""
    total = np.asarray(xq, dtype=np.int64) @ np.asarray(wq, dtype=np.int64).T
    z = total * np.asarray(sw, dtype=np.float64)[None] * np.asarray(sx, dtype=np.float64)[:, None]
    if bias is not None:
        z = z + np.asarray(bias, dtype=np.float64)
    y = ol.act(name, z)
    return (y if residual is None else y + np.asarray(residual, dtype=np.float64)), z
