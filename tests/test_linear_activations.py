"""The dense linear layers' activations and slopes, value by value: exact
arguments (one product with 1, the rest with 0), every finite number of the
type, a relative bound down to fp32's smallest normal numbers.

The bounds, in fp32 steps of 2^-24: e^a is off by its argument's rounding (|a|
steps per rounding of a) and two steps, a reciprocal by two, a product or sum
by one.
- silu: a = z exactly; at most |z| + 8 steps of the value.
- gelu: a = z^2 / 2, exact for 11-bit z; the fitted erfcx is good to 4.5e-7 (8
  steps), its argument's 4 steps count at most 3 times (slope of log erfcx
  against log t), its Horner scheme 8 terms: z^2 / 2 + 32 steps.
- gelu_tanh: a = 2 sqrt(2/pi) (z + 0.044715 z^3) with 6 roundings: 6 |a| + 8.
- A slope's two terms are off by as many steps each, and by one more step of
  1 - s times what multiplies it.
A sigma or exponential below 2^-126 may be taken as 0: 2^-126 times what
multiplies it is allowed absolutely (gelu_tanh's slope: 1 + |z| 2 sqrt(2/pi)
(1 + 0.134145 z^2), 222 at -10, where sigma is 2^-126)."""

import math
import os
import re

import numpy as np
import pytest
import torch

from oracle import linear as ol

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
S = 2.0**-24
C = math.sqrt(2 / math.pi)
SMOOTH = ("silu", "gelu", "gelu_tanh")
TYPES = [torch.float16, torch.bfloat16]


def every(dtype, most):
    """Every number of the type up to ``most`` in magnitude, 16 to a row."""
    z = torch.arange(-(1 << 15), 1 << 15, dtype=torch.int32).to(torch.int16).view(dtype)
    z = z[z.abs() <= most]
    return torch.cat([z, z[: -len(z) % 16]]).reshape(-1, 16)


def steps(act, z):
    if act == "silu":
        return np.abs(z) + 8
    if act == "gelu":
        return z * z / 2 + 32
    return 6 * 2 * C * np.abs(z + 0.044715 * z**3) + 8


def bound(want, err, dtype):
    u = torch.finfo(dtype).eps / 2
    # subnormal results: half of their step
    least = 2.0**-25 if dtype == torch.float16 else 2.0**-134
    return u * np.abs(want) + (1 + u) * err + least


def check(got, want, err, dtype):
    got = got.double().cpu().numpy()
    assert np.isfinite(got).all()
    bad = np.abs(got - want) > bound(want, err, dtype)
    assert not bad.any(), (int(bad.sum()), got[bad][:4], want[bad][:4])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES, ids=["fp16", "bf16"])
@pytest.mark.parametrize("act", SMOOTH)
@pytest.mark.parametrize("rows", [1, 64, 1 << 20])
def test_values(act, dtype, rows):
    import sparse_input_gemv_amd as sa

    x = every(dtype, 100.0).cuda()
    if rows == 1:  # a call each: one row in twenty, all rows of the tail
        keep = (x.abs() < 14).all(1) & (x.abs() > 2).all(1)
        x = x[keep | (torch.arange(len(x), device="cuda") % 20 == 0)]
    eye = torch.eye(16, dtype=dtype, device="cuda")
    one = torch.ones(16, 16, dtype=dtype, device="cuda")  # up projection: the row's sum
    z = x.double().cpu().numpy()
    want = ol.act(act, z)
    err = steps(act, z) * S * np.abs(want) + np.abs(z) * 2.0**-126
    y = torch.cat([sa.dense_linear(x[i:i + rows], eye, act=act) for i in range(0, len(x), rows)])
    check(y, want, err, dtype)
    ux = torch.zeros_like(x)
    ux[:, 0] = 1
    both = torch.cat([x, ux], 1)  # g = x, u = 1
    wg, wu = torch.cat([eye, 0 * eye]), torch.cat([0 * one, one])
    h = torch.cat([sa.gated_linear(both[i:i + rows], wg, wu, act=act) for i in range(0, len(x), rows)])
    assert torch.equal(h, y)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES, ids=["fp16", "bf16"])
@pytest.mark.parametrize("act", SMOOTH)
def test_slopes(act, dtype):
    """dbias of one row is the fp32 slope, rounded once."""
    import sparse_input_gemv_amd as sa

    pre = every(dtype, 100.0).reshape(1, -1).cuda()
    n = pre.shape[1]
    wt = torch.zeros(8, n, dtype=dtype, device="cuda")
    x = torch.zeros(1, 8, dtype=dtype, device="cuda")
    db = sa.dense_linear_backward(torch.ones_like(pre), x, wt, act=act, pre=pre, with_dx=False, with_dwt=False,
                                  with_dbias=True)[2]
    z = pre.double().cpu().numpy()[0]
    k = np.ones_like(z)
    if act == "silu":
        s = ol._sigma(z)
        terms, of = s + np.abs(z) * s * ol._sigma(-z), np.abs(z) * s
    elif act == "gelu":
        s = 0.5 * ol._erfc(-z / math.sqrt(2))
        terms, of = s + np.abs(z) * np.exp(-z * z / 2) / math.sqrt(2 * math.pi), 0 * z
    else:
        a = 2 * C * (z + 0.044715 * z**3)
        s, k = ol._sigma(a), 2 * C * (1 + 0.134145 * z * z)
        terms, of = s + s * ol._sigma(-a) * np.abs(z) * k, np.where(np.abs(a) < 20, np.abs(z) * k * s, 0)
    err = (steps(act, z) + 8) * S * terms + 2 * S * of + (1 + np.abs(z) * k) * 2.0**-126
    check(db, ol.slope(act, z), err, dtype)


def test_oracle_tails():
    """e^-60 beside 1 vanishes; gelu_tanh's argument at -5 is 2 sqrt(2/pi) 10.589375."""
    assert ol.act("silu", [-60.0])[0] == pytest.approx(-60 * math.exp(-60), rel=1e-14)
    assert ol.slope("silu", [-60.0])[0] == pytest.approx(-59 * math.exp(-60), rel=1e-14)
    assert ol.act("gelu_tanh", [-5.0])[0] == pytest.approx(-5 / (1 + math.exp(2 * C * 10.589375)), rel=1e-14)
    assert ol.slope("gelu_tanh", [-9.0])[0] == pytest.approx(
        math.exp(-2 * C * (9 + 0.044715 * 729)) * (1 - 9 * 2 * C * (1 + 0.134145 * 81)), rel=1e-12)


def test_fitted_erfcx():
    """The polynomial in linear.hip, evaluated in fp32 as there, against erfc."""
    src = open(os.path.join(ROOT, "sparse_input_gemv_amd", "csrc", "linear.hip")).read()
    body = src[src.index("normal_cdf(float z"):]
    body = body[:body.index("return z < 0.f")]
    f = np.float32
    scale = f(re.search(r"1\.f \+ ([\d.]+)f \* fabsf\(z\)", body)[1])
    q0 = f(re.search(r"float q = ([-\d.e]+)f;", body)[1])
    cs = [f(s + "1") * f(c) for s, c in re.findall(r"q = q \* t ([+-]) ([\d.e-]+)f;", body)]
    assert len(cs) == 8
    z = -np.linspace(0, 12, 200001).astype(f)
    t = f(1) / (f(1) + scale * -z)
    q = np.full_like(z, q0)
    for c in cs:
        q = (q.astype(np.float64) * t + c).astype(f)  # fused, as the GPU's
    got = (f(0.5) * t * q).astype(np.float64)  # before the factor e^(-z^2/2)
    z64 = z.astype(np.float64)
    want = 0.5 * ol._erfc(-z64 / math.sqrt(2)) * np.exp(z64 * z64 / 2)
    assert np.max(np.abs(got / want - 1)) < 4.5e-7
