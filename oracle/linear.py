"""Dense linear layers in fp64: the product with its epilogue, the gated pair
of projections, and their gradients.

Written as the definitions, on numpy arrays.  ``wt`` is the transposed weight
``[d_in][d_out]``.  With Phi the normal distribution function and sigma the
logistic function, the activations are relu, relu squared, z sigma(z) (silu),
z Phi(z) (gelu) and its tanh form z sigma(2 sqrt(2/pi) (z + 0.044715 z^3)).
"""

from __future__ import annotations

import math

import numpy as np

__all__ = ["ACTIVATIONS", "act", "slope", "linear", "linear_backward", "gated", "gated_backward"]

ACTIVATIONS = ("none", "relu", "relu2", "silu", "gelu", "gelu_tanh")

_erfc = np.vectorize(math.erfc, otypes=[np.float64])


def _sigma(z):
    e = np.exp(-np.abs(z))  # keeps its relative accuracy in the lower tail
    return np.where(z < 0, e, 1.0) / (1.0 + e)


def _tanh_arg(z):
    return 2.0 * math.sqrt(2.0 / math.pi) * (z + 0.044715 * z**3)


def _f64(a):
    return np.asarray(a, dtype=np.float64)


def act(name: str, z) -> np.ndarray:
    z = _f64(z)
    if name == "none":
        return z
    if name == "relu":
        return np.maximum(z, 0.0)
    if name == "relu2":
        return np.maximum(z, 0.0) ** 2
    if name == "silu":
        return z * _sigma(z)
    if name == "gelu":
        return 0.5 * z * _erfc(-z / math.sqrt(2.0))
    if name == "gelu_tanh":
        return z * _sigma(_tanh_arg(z))
    raise ValueError(name)


def slope(name: str, z) -> np.ndarray:
    """The derivative of ``act`` (0 at the kink of relu)."""
    z = _f64(z)
    if name == "none":
        return np.ones_like(z)
    if name == "relu":
        return (z > 0).astype(np.float64)
    if name == "relu2":
        return 2.0 * np.maximum(z, 0.0)
    if name == "silu":
        s = _sigma(z)
        return s + z * s * _sigma(-z)
    if name == "gelu":
        return 0.5 * _erfc(-z / math.sqrt(2.0)) + z * np.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    if name == "gelu_tanh":
        a = _tanh_arg(z)
        s = _sigma(a)
        return s + z * s * _sigma(-a) * 2.0 * math.sqrt(2.0 / math.pi) * (1.0 + 0.134145 * z * z)
    raise ValueError(name)


def linear(x, wt, bias=None, name="none", residual=None):
    """``(y, pre)``: pre = x W^T + bias, y = act(pre) + residual."""
    pre = _f64(x) @ _f64(wt)
    if bias is not None:
        pre = pre + _f64(bias)
    y = act(name, pre)
    if residual is not None:
        y = y + _f64(residual)
    return y, pre


def linear_backward(dy, x, wt, name="none", pre=None):
    """``(dx, dwt, dbias)`` from dy and the forward pass's pre-activation."""
    d = _f64(dy)
    if name != "none":
        d = d * slope(name, pre)
    return d @ _f64(wt).T, _f64(x).T @ d, d.sum(axis=0)


def gated(x, wgt, wut, name="silu"):
    """``(h, g, u)``: h = act(g) * u."""
    g, u = _f64(x) @ _f64(wgt), _f64(x) @ _f64(wut)
    return act(name, g) * u, g, u


def gated_backward(dh, x, wgt, wut, g, u, name="silu"):
    """``(dx, dwgt, dwut)`` from dh and the forward pass's projections."""
    dg = _f64(dh) * _f64(u) * slope(name, g)
    du = _f64(dh) * act(name, g)
    return dg @ _f64(wgt).T + du @ _f64(wut).T, _f64(x).T @ dg, _f64(x).T @ du
