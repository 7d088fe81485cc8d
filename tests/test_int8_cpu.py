"""Linear layers in 8-bit integers without a GPU: the oracle against hand values
and exact fractions, and the C calls' refusals (host checks that fail before any
HIP call)."""

import os
from fractions import Fraction

import numpy as np
import pytest

from oracle import int8 as oi

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "sparse_input_gemv_amd", "libsparse_act.so")
OK, INVALID, UNSUPPORTED, WORKSPACE = range(4)
P = 1 << 20  # aligned, never dereferenced
BIG = 1 << 40
needs_lib = pytest.mark.skipif(not os.path.exists(LIB), reason="library not built")


def test_hand_values():
    q, s = oi.quantize([[127.0, -63.5, 0.5, 1.5, -2.5, 0.0], [0.0] * 6, [np.inf, 1, 2, 3, 4, 5], [np.nan, 1, 2, 3, 4, 5]])
    assert q[0].tolist() == [127, -64, 0, 2, -2, 0] and s[0] == 1.0
    assert not q[1:].any() and s[1] == 0 and np.isnan(s[2:]).all()
    y, z = oi.linear([[1, -2], [3, 4]], [0.5, 2.0], [[10, 20], [-1, 1], [0, 127]], [1.0, 2.0, 0.25], [0.0, 1.0, 0.0], "relu",
                     [[1.0] * 3] * 2)
    assert z.tolist() == [[-15.0, -2.0, -31.75], [220.0, 5.0, 254.0]] and y[0].tolist() == [1.0, 1.0, 1.0]


def exact_code(x, s):
    f = Fraction(float(x)) / Fraction(float(s))
    n = f.numerator // f.denominator
    d = f - n
    return n + (d > Fraction(1, 2) or (d == Fraction(1, 2) and n % 2 == 1))


@pytest.mark.parametrize("bits", [11, 8])
def test_codes_against_exact_fractions(bits):
    rng = np.random.default_rng(3)
    x = np.ldexp(rng.integers(-2**bits + 1, 2**bits, (60, 40)).astype(float), rng.integers(-20, -8, (60, 40)))
    q, s = oi.quantize(x)
    for r in range(60):
        assert s[r] == np.float32(np.abs(x[r]).max()) / np.float32(127)
        assert q[r].tolist() == [exact_code(v, s[r]) for v in x[r]]


@pytest.fixture(scope="module")
def sa():
    import sparse_input_gemv_amd as m
    return m.lib()


def tokens(sa, dtype=0, x=P, ldx=64, T=3, d=64, xq=2 * P, ldq=64, sx=3 * P):
    return sa.act_quantize_int8(dtype, x, ldx, T, d, xq, ldq, sx, None)


def channels(sa, dtype=0, wt=P, ldw=40, d_in=64, d_out=40, wq=2 * P, ldq=64, sw=3 * P, ws=4 * P, wsb=BIG):
    return sa.weight_quantize_int8(dtype, wt, ldw, d_in, d_out, wq, ldq, sw, ws, wsb, None)


def linear(sa, dtype=0, x=P, ldx=64, sx=6 * P, T=3, wq=2 * P, ldw=64, sw=3 * P, d_in=64, d_out=40, bias=None, act=0, res=None,
           ldr=40, y=5 * P, ldy=40, ws=4 * P, wsb=BIG):
    return sa.int8_linear(dtype, x, ldx, sx, T, wq, ldw, sw, d_in, d_out, bias, act, res, ldr, y, ldy, ws, wsb, None)


@needs_lib
@pytest.mark.parametrize("bad, status", [
    (dict(dtype=2), INVALID), (dict(T=-1), INVALID), (dict(T=(1 << 22) + 1), UNSUPPORTED), (dict(d=56), INVALID),
    (dict(d=0), INVALID), (dict(d=131088, ldx=131088, ldq=131088), UNSUPPORTED), (dict(x=None), INVALID),
    (dict(xq=None), INVALID), (dict(sx=None), INVALID), (dict(x=P + 8), INVALID), (dict(xq=P + 8), INVALID),
    (dict(sx=3 * P + 2), INVALID), (dict(ldx=56), INVALID), (dict(ldq=48), INVALID), (dict(ldq=72), INVALID),
    (dict(ldq=1 << 22), UNSUPPORTED), (dict(xq=P), INVALID), (dict(sx=P), INVALID), (dict(sx=2 * P), INVALID)])
def test_token_refusals(sa, bad, status):
    assert tokens(sa, **bad) == status
    assert b"act_quantize_int8" in sa.sa_last_error()


@needs_lib
@pytest.mark.parametrize("bad, status", [
    (dict(dtype=-1), INVALID), (dict(d_in=72), INVALID), (dict(d_out=36), INVALID), (dict(wt=None), INVALID),
    (dict(wq=None), INVALID), (dict(sw=None), INVALID), (dict(ldw=32), INVALID), (dict(ldq=40), INVALID),
    (dict(ws=None), WORKSPACE), (dict(wsb=0), WORKSPACE), (dict(wq=P), INVALID), (dict(sw=2 * P), INVALID)])
def test_channel_refusals(sa, bad, status):
    assert channels(sa, **bad) == status
    assert b"weight_quantize_int8" in sa.sa_last_error()


@needs_lib
@pytest.mark.parametrize("bad, status", [
    (dict(dtype=2), INVALID), (dict(act=6), INVALID), (dict(T=-1), INVALID), (dict(d_in=72), INVALID),
    (dict(d_out=36), INVALID), (dict(d_in=131088, ldx=131088, ldw=131088), UNSUPPORTED), (dict(x=None), INVALID),
    (dict(wq=None), INVALID), (dict(sw=None), INVALID), (dict(y=None), INVALID), (dict(ldx=72), INVALID),
    (dict(ldw=48), INVALID), (dict(sx=6 * P + 2), INVALID), (dict(x=P + 8), INVALID), (dict(bias=P + 8), INVALID),
    (dict(res=7 * P, ldr=32), INVALID), (dict(y=P), INVALID), (dict(y=2 * P), INVALID), (dict(y=3 * P), INVALID),
    (dict(y=6 * P), INVALID), (dict(bias=5 * P), INVALID), (dict(sx=None, ldx=60), INVALID)])
def test_linear_refusals(sa, bad, status):
    assert linear(sa, **bad) == status
    assert b"int8_linear" in sa.sa_last_error()


@needs_lib
def test_workspaces_and_empty_calls(sa):
    # one token of either kind needs none; more 16-bit tokens need room for their codes and scales
    assert sa.int8_linear_workspace_bytes(1, 4096, 4096, 0) == sa.int8_linear_workspace_bytes(1, 4096, 4096, 1) == 0
    need = sa.int8_linear_workspace_bytes(4, 4096, 4096, 0)
    assert need >= 4 * 4096 + 16 and sa.int8_linear_workspace_bytes(4, 4096, 4096, 1) == 0
    kw = dict(T=4, d_in=4096, d_out=4096, ldx=4096, ldw=4096, ldy=4096, sx=None)
    assert linear(sa, **kw, wsb=need - 1) == WORKSPACE and linear(sa, **kw, ws=None) == WORKSPACE
    assert sa.int8_linear_workspace_bytes(0, 4096, 4096, 0) == sa.int8_linear_workspace_bytes(4, 4104, 4096, 0) == 0
    assert linear(sa, T=0, x=None, y=None) == OK and tokens(sa, T=0, x=None, xq=None, sx=None) == OK
    assert linear(sa, T=0, x=None, y=None, sx=None) == OK
