"""Linear layers grouped by expert without a GPU: the fp64 oracle against hand
values and differences, and the C calls' refusals (host checks that fail before
any HIP call)."""

import os

import numpy as np
import pytest

from oracle import grouped as og

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "sparse_input_gemv_amd", "libsparse_act.so")
OK, INVALID, UNSUPPORTED, WORKSPACE = range(4)
P = 1 << 20  # aligned, never dereferenced
BIG = 1 << 40  # a workspace size no check refuses
needs_lib = pytest.mark.skipif(not os.path.exists(LIB), reason="library not built")


def test_hand_values():
    x = np.array([[1.0, 2.0], [3.0, 4.0], [5.0, 6.0], [9.0, 9.0]])
    wt = np.array([[[1.0], [1.0]], [[0.0], [0.0]], [[1.0], [-1.0]]])
    y, pre = og.linear(x, wt, [0, 1, 1, 3], np.array([[0.5], [7.0], [0.0]]), "relu")
    assert list(pre[:3, 0]) == [3.5, -1.0, -1.0] and list(y[:3, 0]) == [3.5, 0.0, 0.0]
    assert np.isnan(y[3, 0])  # no expert's row
    dx, dwt, db = og.linear_backward(np.ones((4, 1)), x, wt, [0, 1, 1, 3])
    assert dx[:3].tolist() == [[1.0, 1.0], [1.0, -1.0], [1.0, -1.0]]
    assert dwt[:, :, 0].tolist() == [[1.0, 2.0], [0.0, 0.0], [8.0, 10.0]] and db[:, 0].tolist() == [1.0, 0.0, 2.0]


def test_clean_offsets():
    assert og.clean_offsets([-3, 5, 2, 99, 7], 8).tolist() == [0, 5, 5, 8, 8]
    assert og.clean_offsets([2, 2, 6], 8).tolist() == [2, 2, 6]


@pytest.mark.parametrize("name", ["none", "relu2", "silu", "gelu", "gelu_tanh"])
def test_gradients_against_differences(name):
    # directional derivative of <dy, f> by central differences in fp64
    rng = np.random.default_rng(7)
    off = [0, 2, 2, 7]
    x, wt, wu = rng.standard_normal((7, 6)), rng.standard_normal((3, 6, 4)), rng.standard_normal((3, 6, 4))
    b, dy = rng.standard_normal((3, 4)), rng.standard_normal((7, 4))
    ex, ew, eu, eb = (rng.standard_normal(a.shape) for a in (x, wt, wu, b))
    h = 1e-6

    def f(s):
        return float((dy * og.linear(x + s * ex, wt + s * ew, off, b + s * eb, name)[0]).sum())

    dx, dwt, db = og.linear_backward(dy, x, wt, off, name, og.linear(x, wt, off, b, name)[1])
    assert (f(h) - f(-h)) / (2 * h) == pytest.approx((dx * ex).sum() + (dwt * ew).sum() + (db * eb).sum(), rel=1e-6, abs=1e-6)

    def fg(s):
        return float((dy * og.gated(x + s * ex, wt + s * ew, wu + s * eu, off, name)[0]).sum())

    _, g, u = og.gated(x, wt, wu, off, name)
    dx, dg, du = og.gated_backward(dy, x, wt, wu, off, g, u, name)
    assert (fg(h) - fg(-h)) / (2 * h) == pytest.approx((dx * ex).sum() + (dg * ew).sum() + (du * eu).sum(), rel=1e-6, abs=1e-6)


@pytest.fixture(scope="module")
def sa():
    import sparse_input_gemv_amd as m
    return m.lib()


def linear(sa, dtype=0, x=P, ldx=64, T=3, wt=2 * P, ldw=32, sw=2048, experts=4, offsets=6 * P, d_in=64, d_out=32,
           bias=None, act=0, res=None, ldr=32, y=3 * P, ldy=32, pre=None, ldpre=32, ws=4 * P, wsb=BIG):
    return sa.grouped_linear(dtype, x, ldx, T, wt, ldw, sw, experts, offsets, d_in, d_out, bias, act, res, ldr, y, ldy,
                             pre, ldpre, ws, wsb, None)


def gated(sa, x=P, ldx=64, T=3, wg=2 * P, wu=5 * P, ldw=32, sw=2048, experts=4, offsets=6 * P, d_in=64, d_out=32, act=3,
          h=3 * P, g=None, u=None, wsb=BIG):
    return sa.grouped_gated_linear(1, x, ldx, T, wg, ldw, sw, wu, ldw, sw, experts, offsets, d_in, d_out, act, h, 32, g,
                                   32, u, 32, 4 * P, wsb, None)


def backward(sa, dtype=1, dy=P, x=2 * P, T=3, wt=3 * P, ldw=32, sw=2048, experts=4, offsets=6 * P, d_in=64, d_out=32,
             act=0, pre=None, dx=7 * P, lddx=64, dwt=8 * P, lddw=32, sdw=2048, dbias=None, wsb=BIG):
    return sa.grouped_linear_backward(dtype, dy, 32, x, 64, T, wt, ldw, sw, experts, offsets, d_in, d_out, act, pre, 32,
                                      dx, lddx, dwt, lddw, sdw, dbias, 4 * P, wsb, None)


def gated_backward(sa, dh=P, x=2 * P, T=3, wg=3 * P, wu=10 * P, experts=4, offsets=6 * P, g=11 * P, u=12 * P, dx=7 * P,
                   dwg=8 * P, dwu=9 * P, lddw=32, sdw=2048, wsb=BIG):
    return sa.grouped_gated_linear_backward(1, dh, 32, x, 64, T, wg, 32, 2048, wu, 32, 2048, experts, offsets, 64, 32, 3,
                                            g, 32, u, 32, dx, 64, dwg, lddw, sdw, dwu, lddw, sdw, 4 * P, wsb, None)


COMMON = [(dict(T=-1), INVALID), (dict(T=(1 << 22) + 1), UNSUPPORTED), (dict(experts=0), INVALID),
          (dict(experts=-1), INVALID), (dict(experts=513), UNSUPPORTED), (dict(offsets=None), INVALID),
          (dict(offsets=6 * P + 2), INVALID), (dict(x=None), INVALID), (dict(x=P + 8), INVALID)]


@needs_lib
@pytest.mark.parametrize("bad, status", COMMON + [
    (dict(dtype=2), INVALID), (dict(act=6), INVALID), (dict(d_in=60), INVALID), (dict(d_out=36), INVALID),
    (dict(wt=None), INVALID), (dict(y=None), INVALID), (dict(ldw=24), INVALID), (dict(sw=-8), INVALID),
    (dict(sw=2052), INVALID), (dict(sw=(1 << 42) + 8), UNSUPPORTED), (dict(bias=P + 8), INVALID),
    (dict(res=9 * P, ldr=24), INVALID), (dict(y=P), INVALID), (dict(y=2 * P), INVALID), (dict(pre=3 * P), INVALID),
    (dict(bias=3 * P), INVALID), (dict(res=7 * P, pre=7 * P), INVALID)])
def test_linear_refusals(sa, bad, status):
    assert linear(sa, **bad) == status
    assert b"grouped_linear" in sa.sa_last_error()


@needs_lib
@pytest.mark.parametrize("bad, status", COMMON + [
    (dict(act=-1), INVALID), (dict(wg=None), INVALID), (dict(wu=None), INVALID), (dict(g=9 * P), INVALID),
    (dict(h=P), INVALID), (dict(h=5 * P), INVALID), (dict(g=9 * P, u=9 * P), INVALID), (dict(sw=12), INVALID)])
def test_gated_refusals(sa, bad, status):
    assert gated(sa, **bad) == status
    assert b"grouped_gated_linear" in sa.sa_last_error()


@needs_lib
@pytest.mark.parametrize("bad, status", COMMON[:7] + [
    (dict(dy=None), INVALID), (dict(x=None), INVALID), (dict(wt=None), INVALID), (dict(act=3), INVALID),
    (dict(dbias=P + 4), INVALID), (dict(dx=P), INVALID), (dict(dwt=2 * P), INVALID), (dict(dx=8 * P), INVALID),
    (dict(dbias=8 * P), INVALID), (dict(dbias=7 * P), INVALID), (dict(lddx=56), INVALID),
    (dict(sdw=2040), INVALID),             # experts one after another would overlap
    (dict(sdw=32, lddw=120), INVALID),     # and as column blocks: four blocks of 32 need 128
    (dict(sdw=0), INVALID)])
def test_backward_refusals(sa, bad, status):
    assert backward(sa, **bad) == status
    assert b"grouped_linear_backward" in sa.sa_last_error()


@needs_lib
@pytest.mark.parametrize("bad, status", COMMON[:7] + [
    (dict(dh=None), INVALID), (dict(g=None), INVALID), (dict(u=None), INVALID), (dict(dwg=None), INVALID),
    (dict(dwu=8 * P), INVALID), (dict(dx=11 * P), INVALID), (dict(sdw=2040), INVALID)])
def test_gated_backward_refusals(sa, bad, status):
    assert gated_backward(sa, **bad) == status
    assert b"grouped_gated_linear_backward" in sa.sa_last_error()


@needs_lib
def test_workspaces(sa):
    need = sa.grouped_linear_workspace_bytes(1, 8, 4096, 4096)
    assert need > 0  # one row: partial sums
    kw = dict(T=1, experts=8, d_in=4096, d_out=4096, ldx=4096, ldw=4096, sw=1 << 24, ldy=4096)
    assert linear(sa, **kw, wsb=need - 1) == WORKSPACE and linear(sa, **kw, ws=None) == WORKSPACE
    assert linear(sa, **kw, ws=P + 8) == INVALID
    assert sa.grouped_linear_workspace_bytes(0, 8, 4096, 4096) == 0
    assert sa.grouped_linear_workspace_bytes(1, 513, 4096, 4096) == 0
    # fp16's backward scratch holds bf16's, and grows with what is asked for
    plain = sa.grouped_linear_backward_workspace_bytes(64, 8, 1024, 512, 0, 0)
    assert sa.grouped_linear_backward_workspace_bytes(64, 8, 1024, 512, 3, 1) > plain
    # the split's partial sums belong to shares: the experts' number does not multiply them
    assert sa.grouped_linear_workspace_bytes(1, 512, 4096, 4096) == need


@needs_lib
def test_empty_calls(sa):
    assert linear(sa, T=0, x=None, y=None) == OK
    assert gated(sa, T=0, x=None, h=None) == OK


@needs_lib
def test_plans():
    import sparse_input_gemv_amd as m
    few = m.grouped_plan("gated", 16, 8, 4096, 14336)
    assert few["tile_rows"] == 16 and few["split"] > 0
    many = m.grouped_plan("forward", 8192, 8, 14336, 4096)
    assert many == {"tile_rows": 256, "split": 256}  # of which the last round alone is shared
    for bad in (("dw", 16, 8, 64, 64), ("forward", 16, 0, 64, 64), ("forward", 16, 8, 60, 64)):
        with pytest.raises(m.SparseActError):
            m.grouped_plan(*bad)
    m.set_linear_tuning(2, 64)
    try:
        assert m.grouped_plan("dx", 500, 4, 1024, 1024) == {"tile_rows": 64, "split": 64}
    finally:
        m.set_linear_tuning()
