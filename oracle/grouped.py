"""Linear layers grouped by expert in fp64: the dense definitions (``linear``)
on each expert's rows.

Rows ``offsets[e]`` to ``offsets[e + 1] - 1`` go through ``wt[e]``.  Results of
rows that no expert takes are NaN, so that nothing can be compared with them.
"""

from __future__ import annotations

import numpy as np

from . import linear as ol

__all__ = ["clean_offsets", "parts", "linear", "linear_backward", "gated", "gated_backward"]


def clean_offsets(offsets, T: int) -> np.ndarray:
    """What offsets of any values count as: within 0 .. T, and at least as
    large as the largest before them."""
    return np.maximum.accumulate(np.clip(np.asarray(offsets, dtype=np.int64), 0, T))


def parts(offsets):
    return [slice(int(a), int(b)) for a, b in zip(offsets[:-1], offsets[1:])]


def _rows(x, cols):
    return np.full((np.shape(x)[0], cols), np.nan)


def linear(x, wt, offsets, bias=None, name="none", residual=None):
    y, pre = _rows(x, wt.shape[2]), _rows(x, wt.shape[2])
    for e, r in enumerate(parts(offsets)):
        y[r], pre[r] = ol.linear(x[r], wt[e], None if bias is None else bias[e], name,
                                 None if residual is None else residual[r])
    return y, pre


def linear_backward(dy, x, wt, offsets, name="none", pre=None):
    E, d_in, d_out = wt.shape
    dx, dwt, dbias = _rows(x, d_in), np.zeros((E, d_in, d_out)), np.zeros((E, d_out))
    for e, r in enumerate(parts(offsets)):
        dx[r], dwt[e], dbias[e] = ol.linear_backward(dy[r], x[r], wt[e], name, None if pre is None else pre[r])
    return dx, dwt, dbias


def gated(x, wgt, wut, offsets, name="silu"):
    h, g, u = (_rows(x, wgt.shape[2]) for _ in range(3))
    for e, r in enumerate(parts(offsets)):
        h[r], g[r], u[r] = ol.gated(x[r], wgt[e], wut[e], name)
    return h, g, u


def gated_backward(dh, x, wgt, wut, offsets, g, u, name="silu"):
    dx, dwg, dwu = _rows(x, wgt.shape[1]), np.zeros(wgt.shape), np.zeros(wut.shape)
    for e, r in enumerate(parts(offsets)):
        dx[r], dwg[e], dwu[e] = ol.gated_backward(dh[r], x[r], wgt[e], wut[e], g[r], u[r], name)
    return dx, dwg, dwu
