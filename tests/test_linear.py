"""Dense linear layers on the GPU (dense_linear, gated_linear and their
gradients) against the fp64 definition.

Two kinds of comparison.  With small integer inputs every sum is exact in
fp32 (below 2^24) in any order, so outputs must equal the correctly rounded
definition bit for bit.  With real inputs an output may be off by half a step
of its type, plus the fp32 sum's error, at most K steps of 2^-23 of the sum of
magnitudes, plus the activation's (a few fp32 steps of its value and
argument)."""

import numpy as np
import pytest
import torch

import sparse_input_gemv_amd as sa
import synthetic as syn
from oracle import gemv as ogemv
from oracle import linear as ol
from oracle import sparsify, swiglu

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
TYPES = [torch.float16, torch.bfloat16]
SMOOTH = ["silu", "gelu", "gelu_tanh"]
# one row to several tiles, odd ones; sizes that end inside a K step, a tile, a 16-column block
ROWS = [1, 2, 5, 16, 17, 31, 33, 64, 65, 100, 129, 257, 300, 515]
DIMS = [(8, 8), (40, 72), (64, 128), (200, 264), (1032, 520), (328, 4104), (4096, 136)]


def ints(shape, lo, hi, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(lo, hi + 1, shape, generator=g).to(dtype).to(DEV)


def same(got, want64):
    want = want64.to(got.dtype)
    assert got.shape == want.shape
    assert torch.equal(got, want), f"{int((got != want).sum())} of {got.numel()} differ"


def relu64(z, act):
    p = z.clamp(min=0)
    return z if act == "none" else p if act == "relu" else p * p


@pytest.mark.parametrize("dims", DIMS, ids=str)
@pytest.mark.parametrize("dtype", TYPES, ids=["fp16", "bf16"])
def test_linear_exact(dims, dtype):
    d_in, d_out = dims
    wt = ints((d_in, d_out), -2, 2, dtype, 1)
    bias = ints((d_out,), -9, 9, dtype, 2)
    for k, t in enumerate(ROWS):
        x = ints((t, d_in), -2, 2, dtype, 10 + t)
        z = x.double() @ wt.double()
        same(sa.dense_linear(x, wt), z)
        act = ("relu", "relu2")[k % 2]
        res = ints((t, d_out), -50, 50, dtype, 3)
        y, pre = sa.dense_linear(x, wt, bias=bias, act=act, residual=res, with_pre=True)
        zb = z + bias.double()
        same(pre, zb)
        same(y, relu64(zb, act) + res.double())
        sa.dense_linear(x, wt, act=act, residual=res, y=res)  # in place on the residual
        same(res, relu64(z, act) + ints((t, d_out), -50, 50, dtype, 3).double())


@pytest.mark.parametrize("dims", DIMS, ids=str)
@pytest.mark.parametrize("dtype", TYPES, ids=["fp16", "bf16"])
def test_gated_exact(dims, dtype):
    d_in, d_out = dims
    wg, wu = ints((d_in, d_out), -2, 2, dtype, 4), ints((d_in, d_out), -1, 1, dtype, 5)
    for k, t in enumerate(ROWS):
        x = ints((t, d_in), -2, 2, dtype, 20 + t)
        act = ("relu", "none")[k % 2]
        h, g, u = sa.gated_linear(x, wg, wu, act=act, with_gu=True)
        g64, u64 = x.double() @ wg.double(), x.double() @ wu.double()
        same(g, g64)
        same(u, u64)
        same(h, relu64(g64, act) * u64)
        assert torch.equal(sa.gated_linear(x, wg, wu, act=act), h)


@pytest.mark.parametrize("dims", DIMS, ids=str)
@pytest.mark.parametrize("dtype", TYPES, ids=["fp16", "bf16"])
def test_linear_backward_exact(dims, dtype):
    d_in, d_out = dims
    wt = ints((d_in, d_out), -2, 2, dtype, 6)
    for k, t in enumerate(ROWS):
        x = ints((t, d_in), -2, 2, dtype, 30 + t)
        dy = ints((t, d_out), -1, 1, dtype, 7)
        pre = ints((t, d_out), -3, 3, dtype, 8)
        act = ("none", "relu", "relu2")[k % 3]
        dx, dwt, db = sa.dense_linear_backward(dy, x, wt, act=act, pre=pre, with_dbias=True)
        p = pre.double().clamp(min=0)
        d = dy.double() * (1.0 if act == "none" else (p > 0).double() if act == "relu" else 2 * p)
        same(dx, d @ wt.double().T)
        same(dwt, x.double().T @ d)
        same(db, d.sum(0))


@pytest.mark.parametrize("dims", DIMS, ids=str)
@pytest.mark.parametrize("dtype", TYPES, ids=["fp16", "bf16"])
def test_gated_backward_exact(dims, dtype):
    d_in, d_out = dims
    wg, wu = ints((d_in, d_out), -2, 2, dtype, 40), ints((d_in, d_out), -1, 1, dtype, 41)
    for t in ROWS:
        x = ints((t, d_in), -2, 2, dtype, 50 + t)
        dh = ints((t, d_out), -1, 1, dtype, 42)
        g, u = ints((t, d_out), -3, 3, dtype, 43), ints((t, d_out), -2, 2, dtype, 44)
        dx, dwg, dwu = sa.gated_linear_backward(dh, x, wg, wu, g, u, act="relu")
        dg = dh.double() * u.double() * (g > 0).double()
        du = dh.double() * g.double().clamp(min=0)
        same(dx, dg @ wg.double().T + du @ wu.double().T)
        same(dwg, x.double().T @ dg)
        same(dwu, x.double().T @ du)


@pytest.fixture
def tuning():
    yield sa.set_linear_tuning
    sa.set_linear_tuning()


@pytest.mark.parametrize("split", [0, 8, 64, 512])
@pytest.mark.parametrize("tile", range(6))
def test_every_tile_and_split(tuning, tile, split):
    """All compiled tiles, whole and shared: ragged rows and columns, K steps
    that end inside a step, shares that cross tiles, more tiles than
    workgroups, every epilogue."""
    tuning(tile, split)
    for t, d_in, d_out, dt in ((1, 200, 72, torch.float16), (77, 584, 392, torch.bfloat16),
                               (530, 328, 1032, torch.float16), (300, 72, 40968, torch.bfloat16)):
        x, res = ints((t, d_in), -2, 2, dt, 90), ints((t, d_out), -50, 50, dt, 91)
        wg, wu = ints((d_in, d_out), -2, 2, dt, 92), ints((d_in, d_out), -1, 1, dt, 93)
        bias = ints((d_out,), -9, 9, dt, 94)
        g64, u64 = x.double() @ wg.double(), x.double() @ wu.double()
        same(sa.dense_linear(x, wg), g64)
        same(sa.dense_linear(x, wg, residual=res), g64 + res.double())
        y, pre = sa.dense_linear(x, wg, bias=bias, act="relu", residual=res, with_pre=True)
        same(pre, g64 + bias.double())
        same(y, (g64 + bias.double()).clamp(min=0) + res.double())
        same(sa.dense_linear(x, wg, bias=bias), g64 + bias.double())
        h, g, u = sa.gated_linear(x, wg, wu, act="relu", with_gu=True)
        same(g, g64)
        same(u, u64)
        same(h, g64.clamp(min=0) * u64)
        same(sa.gated_linear(x, wg, wu, act="relu"), g64.clamp(min=0) * u64)
        dh, u = ints((t, d_out), -1, 1, dt, 95), ints((t, d_out), -1, 1, dt, 96)
        g = ints((t, d_out), -1, 1, dt, 97)
        dx, dwg, dwu = sa.gated_linear_backward(dh, x, wg, wu, g, u, act="relu")
        dg = dh.double() * u.double() * (g > 0).double()
        du = dh.double() * g.double().clamp(min=0)
        same(dx, dg @ wg.double().T + du @ wu.double().T)
        same(dwg, x.double().T @ dg)
        same(dwu, x.double().T @ du)
        dx, dwt, db = sa.dense_linear_backward(dh, x, wg, with_dbias=True)
        same(dx, dh.double() @ wg.double().T)
        same(dwt, x.double().T @ dh.double())
        same(db, dh.double().sum(0))


@pytest.mark.parametrize("shape", [(2000, 4096, 1024), (1024, 1024, 4096), (260, 2056, 11008),
                                   (1, 11008, 4096), (8, 4096, 14336), (48, 14336, 4096),
                                   (2500, 4104, 4168), (4100, 200, 8200)], ids=str)
def test_layer_sizes_exact(shape):
    t, d_in, d_out = shape
    dtype = torch.bfloat16
    x = ints((t, d_in), -2, 2, dtype, 60)
    both = ints((d_in, 2 * d_out), -1, 1, dtype, 61)
    wg, wu = both[:, :d_out], both[:, d_out:]  # side by side
    g64, u64 = x.double() @ wg.double(), x.double() @ wu.double()
    same(sa.dense_linear(x, wg), g64)
    same(sa.gated_linear(x, wg, wu, act="relu"), g64.clamp(min=0) * u64)
    dh, u = ints((t, d_out), -1, 1, dtype, 62), ints((t, d_out), -2, 2, dtype, 63)
    g = ints((t, d_out), -2, 2, dtype, 64)
    dx, dwg, dwu = sa.gated_linear_backward(dh, x, wg, wu, g, u, act="relu")
    dg = dh.double() * u.double() * (g > 0).double()
    du = dh.double() * g.double().clamp(min=0)
    same(dx, dg @ wg.double().T + du @ wu.double().T)
    same(dwg, x.double().T @ dg)
    same(dwu, x.double().T @ du)


# ---- real values -----------------------------------------------------------------

def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def close(got, want, err):
    """|got - want| <= half a step of the result plus ``err`` (before rounding)."""
    g = got.detach().double().cpu().numpy()
    u = half_step(got.dtype)
    tiny = 2.0**-25 if got.dtype == torch.float16 else 0.0  # half a subnormal step
    bad = np.abs(g - want) > u * np.abs(want) + (1 + u) * err + tiny
    assert not bad.any(), f"{int(bad.sum())} of {bad.size}, worst {np.max(np.abs(g - want))}"


E = 2.0**-23


def sum_err(a, b):
    return a.shape[1] * E * (np.abs(a) @ np.abs(b))


def f64(t):
    return t.detach().double().cpu().numpy()


def act_err(z, ez, act):
    """Error of act(z) for an argument off by ez: the slope is below 1.13 for
    the smooth activations; their own evaluation is good to 2^-20 of |z|
    (exp, its argument of at most a few |z|, a reciprocal)."""
    return 1.13 * ez + np.abs(z) * 2.0**-20


@pytest.mark.parametrize("act", SMOOTH)
@pytest.mark.parametrize("dtype", TYPES, ids=["fp16", "bf16"])
@pytest.mark.parametrize("t", [1, 3, 20, 150])
def test_smooth_activations(act, dtype, t):
    d_in, d_out = 264, 200
    gen = torch.Generator().manual_seed(5)
    mk = lambda *s, std=1.0: (torch.randn(*s, generator=gen) * std).to(dtype).to(DEV)  # noqa: E731
    x, wg, wu = mk(t, d_in), mk(d_in, d_out, std=0.15), mk(d_in, d_out, std=0.15)
    bias, res = mk(d_out), mk(t, d_out)
    X, G, U = f64(x), f64(wg), f64(wu)
    y, pre = sa.dense_linear(x, wg, bias=bias, act=act, residual=res, with_pre=True)
    want, wpre = ol.linear(X, G, f64(bias), act, f64(res))
    ez = sum_err(X, G) + 2 * E * np.abs(wpre)
    close(pre, wpre, ez)
    close(y, want, act_err(wpre, ez, act) + 2 * E * np.abs(want))
    h = sa.gated_linear(x, wg, wu, act=act)
    wh, g64, u64 = ol.gated(X, G, U, act)
    eg, eu = sum_err(X, G), sum_err(X, U)
    a = ol.act(act, g64)
    close(h, wh, act_err(g64, eg, act) * (np.abs(u64) + eu) + np.abs(a) * eu + 2 * E * np.abs(wh))


@pytest.mark.parametrize("act", SMOOTH)
@pytest.mark.parametrize("dtype", TYPES, ids=["fp16", "bf16"])
@pytest.mark.parametrize("t", [1, 19, 150])
def test_smooth_gradients(act, dtype, t):
    """Against the formula: d is rounded to the type before the products (half
    a step of each term), slopes are good to 2^-18 (of values up to |z| + 1)."""
    d_in, d_out = 136, 200
    gen = torch.Generator().manual_seed(6)
    mk = lambda *s, std=1.0: (torch.randn(*s, generator=gen) * std).to(dtype).to(DEV)  # noqa: E731
    x, wg, wu = mk(t, d_in), mk(d_in, d_out, std=0.1), mk(d_in, d_out, std=0.1)
    dy, z, u = mk(t, d_out), mk(t, d_out, std=2.0), mk(t, d_out)
    X, G, U, DY, Z, UU = map(f64, (x, wg, wu, dy, z, u))
    h = half_step(dtype)
    sub = 2.0**-25 if dtype == torch.float16 else 0.0

    def rounded(d, scale):  # error of the rounded d: the evaluation's and half a step
        e = scale * (np.abs(Z) + 1) * 2.0**-18
        return e + h * (np.abs(d) + e) + sub

    dx, dwt, db = sa.dense_linear_backward(dy, x, wg, act=act, pre=z, with_dbias=True)
    wdx, wdw, wdb = ol.linear_backward(DY, X, G, act, Z)
    d = DY * ol.slope(act, Z)
    ed = rounded(d, np.abs(DY))
    close(dx, wdx, ed @ np.abs(G).T + sum_err(np.abs(d) + ed, G.T))
    close(dwt, wdw, np.abs(X).T @ ed + sum_err(X.T, np.abs(d) + ed))
    close(db, wdb, (np.abs(DY) * (np.abs(Z) + 1) * 2.0**-18 + (t + 2) * E * np.abs(d)).sum(0))

    dx, dwg, dwu = sa.gated_linear_backward(dy, x, wg, wu, z, u, act=act)
    wdx, wdg, wdu = ol.gated_backward(DY, X, G, U, Z, UU, act)
    dg, du = DY * UU * ol.slope(act, Z), DY * ol.act(act, Z)
    eg, eu = rounded(dg, np.abs(DY * UU)), rounded(du, np.abs(DY))
    close(dx, wdx, eg @ np.abs(G).T + eu @ np.abs(U).T + 2 * sum_err(np.abs(dg) + eg, G.T)
          + 2 * sum_err(np.abs(du) + eu, U.T))
    close(dwg, wdg, np.abs(X).T @ eg + sum_err(X.T, np.abs(dg) + eg))
    close(dwu, wdu, np.abs(X).T @ eu + sum_err(X.T, np.abs(du) + eu))


def test_gradients_against_differences():
    """The gradients along a direction against a central difference of the
    fp64 forward pass; each gradient entry is off by at most a few roundings
    of the terms it sums (3 half steps of the sum of magnitudes)."""
    t, d_in, d_out, act = 37, 72, 88, "silu"
    rng = np.random.default_rng(9)
    to = lambda a: torch.from_numpy(a).to(torch.float16).to(DEV)  # noqa: E731
    x, wg, wu = to(rng.standard_normal((t, d_in))), to(0.1 * rng.standard_normal((d_in, d_out))), \
        to(0.1 * rng.standard_normal((d_in, d_out)))
    dh = to(rng.standard_normal((t, d_out)))
    X, G, U, DH = map(f64, (x, wg, wu, dh))
    _, g, u = sa.gated_linear(x, wg, wu, act=act, with_gu=True)
    dx, dwg, dwu = (f64(v) for v in sa.gated_linear_backward(dh, x, wg, wu, g, u, act=act))
    ex, eg, eu = (rng.standard_normal(a.shape) for a in (X, G, U))
    s = 1e-5
    f = lambda k: float((DH * ol.gated(X + k * ex, G + k * eg, U + k * eu, act)[0]).sum())  # noqa: E731
    num = (f(s) - f(-s)) / (2 * s)
    got = (dx * ex).sum() + (dwg * eg).sum() + (dwu * eu).sum()
    _, g64, u64 = ol.gated(X, G, U, act)
    # g and u arrive rounded: slope and value move by at most 1.13 half steps of |g| + 1 and |u|
    mg = np.abs(DH) * (np.abs(u64) * 1.1 + (np.abs(g64) + 1) * np.abs(u64))
    mu = np.abs(DH) * (np.abs(g64) * 1.13)
    size = ((mg @ np.abs(G).T + mu @ np.abs(U).T) * np.abs(ex)).sum() \
        + ((np.abs(X).T @ mg) * np.abs(eg)).sum() + ((np.abs(X).T @ mu) * np.abs(eu)).sum()
    assert abs(got - num) < 3 * half_step(torch.float16) * size
    assert abs(num) > 100 * abs(got - num)  # and the check says something


# ---- layouts -----------------------------------------------------------------------

def framed(t, pad=24):
    """A copy of ``t`` inside a wider matrix of NaN, and that matrix."""
    rows, cols = t.shape
    big = torch.full((rows + 2, cols + 2 * pad), float("nan"), dtype=t.dtype, device=t.device)
    big[1:-1, pad:-pad] = t
    return big[1:-1, pad:-pad], big


def frame_kept(big, pad=24):
    b = big.clone()
    b[1:-1, pad:-pad] = float("nan")
    return bool(torch.isnan(b).all())


@pytest.mark.parametrize("t", [1, 7, 40, 140, 300])
@pytest.mark.parametrize("dims", [(72, 40), (136, 520), (520, 264)], ids=str)
def test_strided_operands_among_nan(t, dims):
    """Every operand is a window of a matrix of NaN: nothing outside a window
    reaches a result, and nothing outside an output's window is written."""
    d_in, d_out = dims
    dt = torch.float16
    x, wg, wu = ints((t, d_in), -2, 2, dt, 70), ints((d_in, d_out), -2, 2, dt, 71), \
        ints((d_in, d_out), -1, 1, dt, 72)
    dy, z, u = ints((t, d_out), -1, 1, dt, 73), ints((t, d_out), -2, 2, dt, 74), \
        ints((t, d_out), -2, 2, dt, 75)
    win = lambda v: framed(v)[0]  # noqa: E731
    out = lambda r, c: framed(torch.zeros(r, c, dtype=dt, device=DEV))  # noqa: E731
    (y, yb), (pre, pb) = out(t, d_out), out(t, d_out)
    sa.dense_linear(win(x), win(wg), residual=win(z), act="relu", y=y, pre=pre)
    same(pre, x.double() @ wg.double())
    same(y, (x.double() @ wg.double()).clamp(min=0) + z.double())
    assert frame_kept(yb) and frame_kept(pb)
    (h, hb), (g_, gb), (u_, ub) = out(t, d_out), out(t, d_out), out(t, d_out)
    sa.gated_linear(win(x), win(wg), win(wu), act="relu", h=h, g=g_, u=u_)
    same(h, (x.double() @ wg.double()).clamp(min=0) * (x.double() @ wu.double()))
    assert frame_kept(hb) and frame_kept(gb) and frame_kept(ub)
    (dx, dxb), (dwg, dgb), (dwu, dub) = out(t, d_in), out(d_in, d_out), out(d_in, d_out)
    sa.gated_linear_backward(win(dy), win(x), win(wg), win(wu), win(z), win(u), act="relu", dx=dx,
                             dwgt=dwg, dwut=dwu)
    dg = dy.double() * u.double() * (z > 0).double()
    du = dy.double() * z.double().clamp(min=0)
    same(dx, dg @ wg.double().T + du @ wu.double().T)
    same(dwg, x.double().T @ dg)
    same(dwu, x.double().T @ du)
    assert frame_kept(dxb) and frame_kept(dgb) and frame_kept(dub)
    (dx, dxb), (dwt, dwb) = out(t, d_in), out(d_in, d_out)
    _, _, db = sa.dense_linear_backward(win(dy), win(x), win(wg), with_dbias=True, dx=dx, dwt=dwt)
    same(dx, dy.double() @ wg.double().T)
    same(dwt, x.double().T @ dy.double())
    same(db, dy.double().sum(0))
    assert frame_kept(dxb) and frame_kept(dwb)


@pytest.mark.parametrize("t", [5, 150])
def test_gate_and_up_of_different_strides(t):
    dt = torch.bfloat16
    x, dh = ints((t, 200), -2, 2, dt, 76), ints((t, 136), -1, 1, dt, 77)
    wg, wu = framed(ints((200, 136), -2, 2, dt, 78), 16)[0], framed(ints((200, 136), -1, 1, dt, 79), 40)[0]
    g, u = ints((t, 136), -2, 2, dt, 74), framed(ints((t, 136), -2, 2, dt, 75))[0]
    same(sa.gated_linear(x, wg, wu, act="relu"),
         (x.double() @ wg.double()).clamp(min=0) * (x.double() @ wu.double()))
    dx, _, _ = sa.gated_linear_backward(dh, x, wg, wu, g, u, act="relu", with_dw=False)
    dg = dh.double() * u.double() * (g > 0).double()
    du = dh.double() * g.double().clamp(min=0)
    same(dx, dg @ wg.double().T + du @ wu.double().T)


@pytest.mark.parametrize("t", [6, 200])
def test_inf_and_nan_stay_in_their_row(t):
    x, wt = ints((t, 200), -2, 2, torch.float16, 80), ints((200, 72), 1, 2, torch.float16, 81)
    want = sa.dense_linear(x, wt)
    x[1, 3] = float("nan")
    x[4, 199] = float("inf")
    y = sa.dense_linear(x, wt)
    h = sa.gated_linear(x, wt, wt, act="relu")
    assert torch.isnan(y[1]).all() and torch.isinf(y[4]).all()
    assert torch.isnan(h[4] / h[4]).all()
    for act in sa.ACTIVATIONS:
        assert torch.isnan(sa.dense_linear(x, wt, act=act)[1]).all()
        assert torch.isnan(sa.gated_linear(x, wt, wt, act=act)[1]).all()
    keep = [r for r in range(t) if r not in (1, 4)]
    assert torch.equal(y[keep], want[keep]) and torch.isfinite(h[keep]).all()


@pytest.mark.parametrize("act", SMOOTH)
def test_far_arguments(act):
    """Saturated arguments, up to bf16's largest: the value is z or 0 and the
    slope 1 or 0, without Inf or NaN on the way."""
    dt = torch.bfloat16
    z = torch.tensor([[-3e38, -1e20, -1e13, -1e4, -200, 200, 1e4, 1e13, 1e18, 3e38]], dtype=dt, device=DEV)
    z = torch.cat([z, z[:, :6]], 1)  # 16 values
    eye = torch.eye(16, dtype=dt, device=DEV)
    one = torch.ones(1, 16, dtype=dt, device=DEV)
    up = z > 0
    for j in range(16):  # one value at a time: 0 * z of the others stays finite, z * 1 exact
        x = torch.zeros(1, 16, dtype=dt, device=DEV)
        x[0, j] = z[0, j]
        y = sa.dense_linear(x, eye, act=act)
        assert y[0, j] == (z[0, j] if up[0, j] else 0)
    dx, _, db = sa.dense_linear_backward(one, one, eye, act=act, pre=z, with_dbias=True)
    assert torch.equal(dx, up.to(dt)) and torch.equal(db, up[0].to(dt))
    g = sa.gated_linear_backward(one, one, eye, eye, z, torch.zeros_like(one), act=act)[0]
    assert torch.equal(g, torch.where(up, z, 0 * z).to(dt))


def test_no_rows():
    dt = torch.float16
    wt = ints((64, 40), -2, 2, dt, 82)
    x = torch.empty(0, 64, dtype=dt, device=DEV)
    y = torch.empty(0, 40, dtype=dt, device=DEV)
    assert sa.dense_linear(x, wt).shape == (0, 40)
    assert sa.gated_linear(x, wt, wt).shape == (0, 40)
    dx, dwt, db = sa.dense_linear_backward(y, x, wt, act="silu", pre=y, with_dbias=True)
    assert dx.shape == (0, 64) and not dwt.any() and not db.any() and dwt.shape == (64, 40)
    dx, dwg, dwu = sa.gated_linear_backward(y, x, wt, wt, y, y)
    assert dx.shape == (0, 64) and not dwg.any() and not dwu.any()


def test_vectors_and_parts():
    dt = torch.bfloat16
    wt = ints((64, 40), -2, 2, dt, 83)
    x, dy = ints((64,), -2, 2, dt, 84), ints((40,), -1, 1, dt, 85)
    y = sa.dense_linear(x, wt)
    assert y.shape == (40,)
    same(y, x.double() @ wt.double())
    dx, dwt, db = sa.dense_linear_backward(dy, x, wt, with_dwt=False)
    assert dwt is None and db is None
    same(dx, wt.double() @ dy.double())
    dx, dwt, db = sa.dense_linear_backward(dy, x, wt, with_dx=False, with_dbias=True)
    assert dx is None
    same(dwt, x.double()[:, None] * dy.double())
    same(db, dy.double())
    h, g, u = sa.gated_linear(x, wt, wt, with_gu=True)
    assert h.shape == g.shape == u.shape == (40,)


def test_offsets_past_32_bits():
    """Row operands of more than 2^31 entries: the last rows are right."""
    t, d_in, d_out, dt = 140001, 8, 16384, torch.bfloat16
    x, wt = ints((t, d_in), -2, 2, dt, 86), ints((d_in, d_out), -2, 2, dt, 87)
    y = sa.dense_linear(x, wt)
    assert y.numel() > 2**31
    for s in (slice(0, 300), slice(70000, 70300), slice(t - 300, t)):
        same(y[s], x[s].double() @ wt.double())
    y.clamp_(-1, 1)
    dx, dwt, db = sa.dense_linear_backward(y, x, wt, with_dbias=True)
    for s in (slice(0, 300), slice(t - 300, t)):
        same(dx[s], y[s].double() @ wt.double().T)
    want = sum((x[i:i + 20000].double().T @ y[i:i + 20000].double() for i in range(0, t, 20000)))
    same(dwt, want)  # sums below 2^24
    same(db, sum(y[i:i + 20000].double().sum(0) for i in range(0, t, 20000)))


# ---- streams, graphs, repeatability --------------------------------------------------

def layer(x, wg, wu, wd, dy):
    """A gated block with its residual, forward and backward."""
    h, g, u = sa.gated_linear(x, wg, wu, with_gu=True)
    y = sa.dense_linear(h, wd, residual=x)
    dh, dwd, _ = sa.dense_linear_backward(dy, h, wd)
    dx, dwg, dwu = sa.gated_linear_backward(dh, x, wg, wu, g, u)
    return y, dx, dwg, dwu, dwd


def layer_inputs(t, d, ff, seed, dtype=torch.bfloat16):
    gen = torch.Generator().manual_seed(seed)
    mk = lambda *s, std=1.0: (torch.randn(*s, generator=gen) * std).to(dtype).to(DEV)  # noqa: E731
    return mk(t, d), mk(d, ff, std=0.05), mk(d, ff, std=0.05), mk(ff, d, std=0.05), mk(t, d)


@pytest.mark.parametrize("t", [1, 12, 130])
def test_block_forward_and_backward(t):
    """The operators run together as a block, against the fp64 chain: each
    tensor in relative 2-norm within 5 half steps (h, g, u, dh, dg, du and the
    output are each rounded once)."""
    x, wg, wu, wd, dy = layer_inputs(t, 264, 520, 3)
    got = layer(x, wg, wu, wd, dy)
    X, G, U, D, DY = map(f64, (x, wg, wu, wd, dy))
    h, g, u = ol.gated(X, G, U)
    y, _ = ol.linear(h, D, residual=X)
    dh, dwd, _ = ol.linear_backward(DY, h, D)
    want = (y, *ol.gated_backward(dh, X, G, U, g, u), dwd)
    for a, b in zip(got, want):
        assert np.linalg.norm(f64(a) - b) <= 5 * half_step(torch.bfloat16) * np.linalg.norm(b)


@pytest.mark.parametrize("t", [1, 12, 130])
def test_equal_calls_give_equal_bits(t):
    ins = layer_inputs(t, 1032, 2056, 4)
    first = [v.clone() for v in layer(*ins)]
    for _ in range(20):
        for a, b in zip(layer(*ins), first):
            assert torch.equal(a, b)


@pytest.mark.parametrize("t", [1, 40])
def test_graphs_and_streams(t):
    """Two captured graphs of the block replayed on two streams at once, the
    same calls running eagerly on a third: every replay gives the eager bits."""
    a, b = layer_inputs(t, 1032, 2056, 5), layer_inputs(t, 1032, 2056, 6)
    want = [[v.clone() for v in layer(*i)] for i in (a, b)]
    side = torch.cuda.Stream()
    graphs, outs = [], []
    for ins in (a, b):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs.append(layer(*ins))
        graphs.append(gr)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        for o in outs:
            for v in o:
                v.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(s1):
            graphs[0].replay()
        with torch.cuda.stream(s2):
            graphs[1].replay()
        with torch.cuda.stream(side):
            eager = layer(*a)
        torch.cuda.synchronize()
        for o, w in zip(outs + [eager], want + [want[0]]):
            for v, e in zip(o, w):
                assert torch.equal(v, e)


@pytest.mark.parametrize("t", [1, 16, 64])
def test_calls_on_streams_at_once(t):
    """Single-token calls, whose workgroups add their partial sums within the
    launch, on three streams at once: each stream has its own counters and
    scratch, and every call gives the bits of a call by itself."""
    ins = [layer_inputs(t, 2056, 1032, 7 + k, torch.float16) for k in range(3)]
    f = lambda i: (sa.gated_linear(i[0], i[1], i[2], with_gu=True),  # noqa: E731
                   sa.dense_linear(i[0], i[1], bias=i[3][:, 0].contiguous(), act="gelu"))
    want = [f(i) for i in ins]
    streams = [torch.cuda.Stream() for _ in ins]
    torch.cuda.synchronize()
    for _ in range(10):
        got = []
        for _ in range(5):
            for i, s in zip(ins, streams):
                with torch.cuda.stream(s):
                    got.append(f(i))
        torch.cuda.synchronize()
        for k, (gu, y) in enumerate(got):
            for a, b in zip(gu + (y,), want[k % 3][0] + (want[k % 3][1],)):
                assert torch.equal(a, b)


# ---- with the sparse operators --------------------------------------------------------

def test_decode_block_with_the_sparse_down_projection():
    """One token: gate and up in one call, then the down projection over the
    surviving entries of h (threshold) or of g, u (CATS), against the oracles
    on the values this call wrote."""
    d, ff, t = 512, 1376, 0.05
    wg, wu = syn.weight_t(ff, d, 90), syn.weight_t(ff, d, 91)
    wd = syn.weight_t(d, ff, 92)
    x = syn.gaussian_f16((d,), 1.0, 93)
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(DEV)  # noqa: E731
    h, g, u = sa.gated_linear(dev(x), dev(wg), dev(wu), with_gu=True)
    close(h[None], ol.gated(x[None], wg, wu)[0], 1e-4)
    y = sa.sparse_gemv_threshold(dev(wd), h, t)
    keep = sparsify.threshold_sparsify(h.cpu().numpy(), t)[0]
    ref = ogemv.masked_gemv(wd, h.cpu().numpy(), keep)
    assert np.linalg.norm(f64(y) - ref) <= 2e-3 * np.linalg.norm(ref)
    yc, _, _ = sa.masked_swiglu_down(g, u, dev(wd), 0.0, "cats")
    dense = sa.dense_linear(h, dev(wd))  # a threshold of 0 keeps every entry
    assert np.linalg.norm(f64(yc) - f64(dense)) <= 2e-3 * np.linalg.norm(f64(dense))


def test_refusals():
    dt = torch.float16
    x, wt = ints((3, 64), -1, 1, dt, 1), ints((64, 40), -1, 1, dt, 2)
    bad = [
        lambda: sa.dense_linear(x.cpu(), wt), lambda: sa.dense_linear(x.float(), wt.float()),
        lambda: sa.dense_linear(x, wt.bfloat16()), lambda: sa.dense_linear(x, wt[:32]),
        lambda: sa.dense_linear(x, wt, act="tanh"), lambda: sa.dense_linear(x, wt.T.contiguous().T),
        lambda: sa.dense_linear(x, wt, bias=wt[0, :32]), lambda: sa.dense_linear(x, wt, residual=x),
        lambda: sa.dense_linear(x, wt, y=x), lambda: sa.dense_linear(x[None], wt),
        lambda: sa.dense_linear(x, wt.cpu()), lambda: sa.gated_linear(x, wt, wt[:, :32]),
        lambda: sa.gated_linear_backward(x, x, wt, wt, x, x),
        lambda: sa.dense_linear_backward(sa.dense_linear(x, wt), x, wt, act="silu"),
    ]
    for f in bad:
        with pytest.raises(ValueError):
            f()
    for f in (lambda: sa.dense_linear(x[:, :60], wt[:60]),          # d_in not a multiple of 8
              lambda: sa.dense_linear(x[:, 4:60], wt[:56]),         # rows not 16-byte aligned
              lambda: sa.dense_linear(x[:1].expand(3, 64), wt),     # rows on top of each other
              lambda: sa.dense_linear(x, wt[:, :36])):              # d_out not a multiple of 8
        with pytest.raises(sa.SparseActError) as e:
            f()
        assert e.value.status == 1
