"""Dense linear layers without a GPU: the fp64 oracle against hand values and
differences, and the C calls' refusals (host checks that fail before any HIP
call)."""

import math
import os

import numpy as np
import pytest

from oracle import linear as ol

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "sparse_input_gemv_amd", "libsparse_act.so")
OK, INVALID, UNSUPPORTED, WORKSPACE = range(4)
P = 1 << 20  # aligned, never dereferenced
needs_lib = pytest.mark.skipif(not os.path.exists(LIB), reason="library not built")


def test_activation_hand_values():
    # silu(ln 3) = 3/4 ln 3; gelu(1) = Phi(1); relu2(3) = 9; tanh form by its formula
    assert ol.act("silu", [math.log(3)])[0] == pytest.approx(0.75 * math.log(3), rel=1e-15)
    assert ol.act("gelu", [1.0])[0] == pytest.approx(0.8413447460685429, rel=1e-15)
    assert ol.act("gelu", [-8.0])[0] == pytest.approx(-8 * 6.220960574271785e-16, rel=1e-12)
    assert list(ol.act("relu2", [3.0, -3.0, 0.0])) == [9.0, 0.0, 0.0]
    assert list(ol.slope("relu", [2.0, -2.0, 0.0])) == [1.0, 0.0, 0.0]
    assert ol.act("gelu_tanh", [1.0])[0] == pytest.approx(0.8411919906082768, rel=1e-12)


@pytest.mark.parametrize("name", ol.ACTIVATIONS)
def test_slopes_against_differences(name):
    # central differences: truncation h^2/6 |f'''| (|f'''| < 4 here), rounding 2^-52 |f| / h
    z = np.linspace(-4.03, 4.03, 403)
    h = 1e-5
    num = (ol.act(name, z + h) - ol.act(name, z - h)) / (2 * h)
    err = np.abs(num - ol.slope(name, z))
    if name in ("relu", "relu2"):  # at the kink the differences are h / 2h = 1/2 and h^2 / 2h = h/2
        assert z[201] == 0 and err[201] == pytest.approx(0.5 if name == "relu" else h / 2, rel=1e-12)
        err[201] = 0
    assert np.max(err) < 4 * h * h + 2 * 2.0**-52 * 20 / h


def _direction(rng, *arrays):
    return [rng.standard_normal(a.shape) for a in arrays]


@pytest.mark.parametrize("name", ["none", "relu2", "silu", "gelu", "gelu_tanh"])
def test_gradients_against_differences(name):
    # directional derivative of <dy, f> by central differences in fp64
    rng = np.random.default_rng(7)
    x, wt, b = rng.standard_normal((5, 6)), rng.standard_normal((6, 4)), rng.standard_normal(4)
    wu, dy = rng.standard_normal((6, 4)), rng.standard_normal((5, 4))
    ex, ew, eu = _direction(rng, x, wt, wu)
    eb = rng.standard_normal(4)
    h = 1e-6

    def f(s):
        return float((dy * ol.linear(x + s * ex, wt + s * ew, b + s * eb, name)[0]).sum())

    dx, dwt, db = ol.linear_backward(dy, x, wt, name, ol.linear(x, wt, b, name)[1])
    want = (dx * ex).sum() + (dwt * ew).sum() + (db * eb).sum()
    assert (f(h) - f(-h)) / (2 * h) == pytest.approx(want, rel=1e-6, abs=1e-6)

    def fg(s):
        return float((dy * ol.gated(x + s * ex, wt + s * ew, wu + s * eu, name)[0]).sum())

    _, g, u = ol.gated(x, wt, wu, name)
    dx, dg, du = ol.gated_backward(dy, x, wt, wu, g, u, name)
    want = (dx * ex).sum() + (dg * ew).sum() + (du * eu).sum()
    assert (fg(h) - fg(-h)) / (2 * h) == pytest.approx(want, rel=1e-6, abs=1e-6)


@pytest.fixture(scope="module")
def sa():
    import sparse_input_gemv_amd as m
    return m.lib()


BIG = 1 << 40  # a workspace size no check refuses


def linear(sa, dtype=0, x=P, ldx=64, T=3, wt=2 * P, ldw=32, d_in=64, d_out=32, bias=None, act=0,
           res=None, ldr=32, y=3 * P, ldy=32, pre=None, ldpre=32, ws=4 * P, wsb=BIG,
           tk=None):
    return sa.dense_linear(dtype, x, ldx, T, wt, ldw, d_in, d_out, bias, act, res, ldr, y, ldy, pre,
                           ldpre, ws, wsb, tk, None)


@needs_lib
@pytest.mark.parametrize("bad, status", [
    (dict(dtype=2), INVALID), (dict(dtype=-1), INVALID), (dict(act=6), INVALID),
    (dict(act=-1), INVALID), (dict(T=-1), INVALID), (dict(T=(1 << 22) + 1), UNSUPPORTED),
    (dict(d_in=60), INVALID), (dict(d_in=0), INVALID), (dict(d_out=36), INVALID),
    (dict(d_out=(1 << 21) + 8, ldw=(1 << 21) + 8), UNSUPPORTED),
    (dict(x=None), INVALID), (dict(wt=None), INVALID), (dict(y=None), INVALID),
    (dict(x=P + 2), INVALID), (dict(wt=2 * P + 8), INVALID), (dict(y=3 * P + 4), INVALID),
    (dict(bias=P + 8), INVALID), (dict(res=P + 8), INVALID), (dict(pre=P + 8), INVALID),
    (dict(ldx=56), INVALID), (dict(ldx=68), INVALID), (dict(ldw=24), INVALID),
    (dict(ldy=0), INVALID), (dict(res=5 * P, ldr=24), INVALID), (dict(pre=5 * P, ldpre=0), INVALID),
    (dict(ldx=1 << 22), UNSUPPORTED),
    (dict(y=P), INVALID), (dict(y=2 * P), INVALID), (dict(pre=3 * P), INVALID),
    (dict(res=5 * P, pre=5 * P), INVALID), (dict(tk=P + 4), INVALID),
])
def test_dense_linear_refusals(sa, bad, status):
    assert linear(sa, **bad) == status
    assert b"dense_linear" in sa.sa_last_error()


@needs_lib
def test_empty_calls(sa):
    assert linear(sa, T=0, x=None, y=None) == OK
    assert sa.gated_linear(0, None, 64, 0, P, 32, 2 * P, 32, 64, 32, 3, None, 32, None, 0, None, 0,
                           None, 0, None, None) == OK


@needs_lib
def test_workspace_refusals(sa):
    need = sa.dense_linear_workspace_bytes(1, 4096, 4096)
    assert need > 0  # one token splits the input over workgroups
    kw = dict(T=1, d_in=4096, d_out=4096, ldx=4096, ldw=4096, ldy=4096)
    assert linear(sa, **kw, wsb=need - 1) == WORKSPACE
    assert linear(sa, **kw, ws=None) == WORKSPACE
    assert linear(sa, **kw, ws=4 * P + 8, wsb=need) == INVALID
    assert sa.dense_linear_workspace_bytes(1, 4095, 4096) == 0  # invalid sizes
    assert sa.gated_linear_backward_workspace_bytes(100, 64, 32) >= 2 * 100 * 32 * 2
    assert sa.dense_linear_backward_workspace_bytes(100, 64, 32, 9, 0) == 0


def gated(sa, dtype=1, x=P, ldx=64, T=3, wg=2 * P, ldg=32, wu=3 * P, ldu=32, d_in=64, d_out=32,
          act=3, h=4 * P, ldh=32, g=5 * P, ldgo=32, u=6 * P, lduo=32, ws=7 * P, wsb=BIG, tk=None):
    return sa.gated_linear(dtype, x, ldx, T, wg, ldg, wu, ldu, d_in, d_out, act, h, ldh, g, ldgo, u,
                           lduo, ws, wsb, tk, None)


@needs_lib
@pytest.mark.parametrize("bad, status", [
    (dict(dtype=7), INVALID), (dict(act=7), INVALID), (dict(wg=None), INVALID),
    (dict(wu=None), INVALID), (dict(h=None), INVALID), (dict(g=None), INVALID),
    (dict(u=None), INVALID), (dict(u=P + 2), INVALID), (dict(ldu=16), INVALID),
    (dict(ldgo=16), INVALID), (dict(lduo=28), INVALID), (dict(h=P), INVALID),
    (dict(h=5 * P), INVALID), (dict(g=6 * P), INVALID), (dict(u=3 * P), INVALID),
    (dict(d_in=12), INVALID), (dict(d_out=4), INVALID), (dict(wu=3 * P + 8), INVALID),
    (dict(tk=P + 8), INVALID),
])
def test_gated_linear_refusals(sa, bad, status):
    assert gated(sa, **bad) == status
    assert b"gated_linear" in sa.sa_last_error()


def linear_bwd(sa, dtype=0, dy=P, lddy=32, x=2 * P, ldx=64, T=3, wt=3 * P, ldw=32, d_in=64,
               d_out=32, act=3, pre=4 * P, ldpre=32, dx=5 * P, lddx=64, dwt=6 * P, lddwt=32,
               db=None, ws=7 * P, wsb=BIG):
    return sa.dense_linear_backward(dtype, dy, lddy, x, ldx, T, wt, ldw, d_in, d_out, act, pre,
                                    ldpre, dx, lddx, dwt, lddwt, db, ws, wsb, None)


@needs_lib
@pytest.mark.parametrize("bad, status", [
    (dict(dy=None), INVALID), (dict(x=None), INVALID), (dict(wt=None), INVALID),
    (dict(pre=None), INVALID), (dict(dx=5 * P + 2), INVALID), (dict(lddx=32), INVALID),
    (dict(lddwt=24), INVALID), (dict(db=P + 2), INVALID), (dict(dx=P), INVALID),
    (dict(dx=4 * P), INVALID), (dict(dwt=3 * P), INVALID), (dict(dwt=5 * P), INVALID),
    (dict(ws=None), WORKSPACE), (dict(wsb=100), WORKSPACE), (dict(db=2 * P), INVALID),
])
def test_dense_linear_backward_refusals(sa, bad, status):
    assert linear_bwd(sa, **bad) == status
    assert b"dense_linear_backward" in sa.sa_last_error()


def gated_bwd(sa, dtype=0, dh=P, lddh=32, x=2 * P, ldx=64, T=3, wg=3 * P, ldwg=32, wu=4 * P,
              ldwu=32, d_in=64, d_out=32, act=3, g=5 * P, ldg=32, u=6 * P, ldu=32, dx=7 * P,
              lddx=64, dwg=8 * P, lddwg=32, dwu=9 * P, lddwu=32, ws=10 * P, wsb=BIG):
    return sa.gated_linear_backward(dtype, dh, lddh, x, ldx, T, wg, ldwg, wu, ldwu, d_in, d_out,
                                    act, g, ldg, u, ldu, dx, lddx, dwg, lddwg, dwu, lddwu, ws, wsb,
                                    None)


@needs_lib
@pytest.mark.parametrize("bad, status", [
    (dict(dh=None), INVALID), (dict(g=None), INVALID), (dict(u=None), INVALID),
    (dict(dwg=None), INVALID), (dict(dwu=None), INVALID), (dict(x=None), INVALID),
    (dict(wg=None), INVALID), (dict(lddwu=8), INVALID), (dict(dx=6 * P), INVALID),
    (dict(dwu=8 * P), INVALID), (dict(dwg=2 * P), INVALID), (dict(ws=None), WORKSPACE),
    (dict(wsb=64), WORKSPACE), (dict(T=-3), INVALID),
])
def test_gated_linear_backward_refusals(sa, bad, status):
    assert gated_bwd(sa, **bad) == status
    assert b"gated_linear_backward" in sa.sa_last_error()


def plan(sa, op, t, d_in, d_out):
    import ctypes
    o = [ctypes.c_int() for _ in range(3)] + [ctypes.c_int64()]
    assert sa.sa_linear_plan(op, t, d_in, d_out, *[ctypes.addressof(v) for v in o]) == OK
    return tuple(v.value for v in o)  # rows, cols, split, tiles


@needs_lib
def test_plans(sa):
    """Large products take whole 256 x 256 tiles, few rows share the weights'
    steps over one workgroup per CU, and the workspace holds the partials."""
    assert plan(sa, 0, 8192, 14336, 4096) == (256, 256, 0, 512)
    assert plan(sa, 1, 8192, 4096, 14336) == (256, 128, 0, 3584)
    assert plan(sa, 3, 4096, 4096, 11008) == (256, 256, 0, 688)
    assert plan(sa, 5, 4096, 4096, 11008) == (256, 256, 0, 1376)
    rows, cols, split, tiles = plan(sa, 0, 1, 4096, 4096)
    assert (rows, split) == (16, 256) and tiles == 32
    # 64 steps x 32 tiles over 256 shares: 8 steps each, 8 shares per tile
    assert sa.dense_linear_workspace_bytes(1, 4096, 4096) == 8 * 4096 * 4
    rows, cols, split, tiles = plan(sa, 1, 1, 4096, 11008)
    assert (rows, split, tiles) == (16, 256, 86)
    # 21.5 steps per share: a tile of 64 steps meets at most 5 shares
    assert sa.gated_linear_workspace_bytes(1, 4096, 11008) in (4 * 11008 * 8, 5 * 11008 * 8)
    assert sa.sa_linear_plan(6, 1, 64, 64, P, P, P, P) == INVALID
    assert sa.sa_linear_plan(0, 1, 60, 64, P, P, P, P) == INVALID
    assert sa.sa_linear_plan(0, 1, 64, 64, None, P, P, P) == INVALID
    assert sa.sa_set_linear_tuning(6, 0) == INVALID
    assert sa.sa_set_linear_tuning(0, 513) == INVALID
    assert sa.sa_set_linear_tuning(-2, 0) == INVALID
    assert sa.sa_set_linear_tuning(-1, -1) == OK
