"""fp16 gradients of the layers grouped by expert where d lies outside fp16's
range: by rows' scales for dx, by experts' columns' for dW.

Exact: entries of d are small integers times a power of two of their expert, row
and column, so that d is exact when it is scaled and lost (or infinite) when it
is not, every sum is exact in fp32, and outputs must equal the correctly rounded
definition bit for bit.  Real values: the dense layers' bounds, a column's
largest being that of the expert's own rows."""

import numpy as np
import pytest
import torch

import sparse_input_gemv_amd as sa
from oracle import linear as ol
from test_grouped import by_expert, kept, offsets_of
from test_linear import DEV, E, f64, ints, same
from test_linear import tuning  # noqa: F401
from test_linear_range import close, dev, representable, rounded
from test_grouped_shared import shared

pytestmark = pytest.mark.gpu
F = torch.float16
# an expert's powers of two: of dy (dh), of what d multiplies it with, of x and the weights
SMALL, PLAIN, LARGE = (-16, -8, 13), (0, 0, 0), (11, 3, -12)


def powers(n, lo, hi, seed):
    gen = torch.Generator().manual_seed(seed)
    return torch.exp2(torch.randint(lo, hi + 1, (n,), generator=gen).double()).to(DEV)


def exact_inputs(counts, kinds, d_in, d_out, start, after=3):
    """fp16 tensors dy, x, wg, wu, g, u; rows of no expert are NaN."""
    T, n = start + sum(counts) + after, len(counts)
    s = lambda i: torch.tensor([2.0**k[i] for k in kinds], dtype=torch.float64, device=DEV)  # noqa: E731
    of = torch.full((T,), -1, device=DEV)
    for e, r in by_expert(counts, start):
        of[r] = e
    own = lambda i: torch.where(of < 0, float("nan"), s(i)[of.clamp(min=0)])[:, None]  # noqa: E731
    to = lambda v: v.to(F)  # noqa: E731
    sizes = powers(T, -2, 2, 1)[:, None] * powers(d_out, -2, 2, 2)
    return (to(ints((T, d_out), -1, 1, F, 3).double() * sizes * own(0)), to(ints((T, d_in), -2, 2, F, 4).double() * own(2)),
            to(ints((n, d_in, d_out), -2, 2, F, 5).double() * s(2)[:, None, None]),
            to(ints((n, d_in, d_out), -1, 1, F, 6).double() * s(2)[:, None, None]),
            to(ints((T, d_out), -2, 2, F, 7).double() * own(1)), to(ints((T, d_out), -2, 2, F, 8).double() * own(1)))


def filled(*shape):
    return torch.full(shape, 7, dtype=F, device=DEV)


def check_exact(counts, kinds, d_in, d_out, start=2, with_dw=True):
    dy, x, wg, wu, g, u = exact_inputs(counts, kinds, d_in, d_out, start)
    (T, _), n, off = dy.shape, len(counts), offsets_of(counts, start)
    # ungated, by relu2: d = dy 2 max(g, 0)
    dx = filled(T, d_in)
    _, dwt, db = sa.grouped_linear_backward(dy, x, wg, off, act="relu2", pre=g, with_dbias=with_dw, with_dwt=with_dw, dx=dx)
    kept(dx, 7, counts, start)
    gx = filled(T, d_in)
    _, dwg, dwu = sa.grouped_gated_linear_backward(dy, x, wg, wu, off, g, u, act="relu", with_dw=with_dw, dx=gx)
    kept(gx, 7, counts, start)
    seen = []
    for e in range(n):
        o = off.tolist()
        r = slice(o[e], o[e + 1])
        D, X, G, U, P = (v[r].double() for v in (dy, x, g, u, g))
        d, dg, du = D * 2 * P.clamp(min=0), D * U * (G > 0), D * G.clamp(min=0)
        same(dx[r], d @ wg[e].double().T)
        same(gx[r], dg @ wg[e].double().T + du @ wu[e].double().T)
        if with_dw:
            same(dwt[e], X.T @ d)
            same(db[e], d.sum(0))
            same(dwg[e], X.T @ dg)
            same(dwu[e], X.T @ du)
        if r.stop > r.start:
            seen += [dg.abs().max().item(), du.abs().max().item()]
    return seen


RAGGED = [0, 40, 1, 300, 0, 90, 37, 2, 0]
KINDS = [PLAIN, SMALL, LARGE, PLAIN, SMALL, LARGE, SMALL, PLAIN, LARGE]


@pytest.mark.parametrize("dims", [(8, 8), (40, 72), (200, 264), (72, 1032), (584, 392)], ids=str)
def test_exact(dims):
    seen = check_exact(RAGGED, KINDS, *dims)
    if dims[1] > 64:  # enough values that both ends occur
        assert max(seen) > 65504 and min(seen) < 2.0**-18


@pytest.mark.parametrize("kind", [SMALL, LARGE], ids=["small", "large"])
@pytest.mark.parametrize("counts", [[37], [0, 1], [70, 0, 0, 513]], ids=str)
def test_exact_all_experts_alike(counts, kind):
    check_exact(counts, [kind] * len(counts), 136, 264)


@pytest.mark.parametrize("split", [0, 8, 64, 256])
@pytest.mark.parametrize("tile", range(5))
def test_exact_in_every_tile_and_split(tuning, tile, split):  # noqa: F811
    tuning(tile, split)
    check_exact(RAGGED, KINDS, 584, 392)
    check_exact([1], [SMALL], 200, 584)
    check_exact([530, 3, 260], [LARGE, SMALL, PLAIN], 328, 1032)


def test_exact_in_a_shared_rest():
    """As planned: 256-row tiles, whole rounds of them and a rest that is shared."""
    counts, kinds = [0, 1300, 0, 700, 257, 1, 2300, 0], [PLAIN, SMALL, PLAIN, LARGE, SMALL, LARGE, PLAIN, LARGE]
    shared("dx", counts, 3848, 2824)
    shared("gated_dx", counts, 3848, 2824)
    check_exact(counts, kinds, 3848, 2824, with_dw=False)


def test_one_gradient_alone_has_the_bits_of_both():
    counts = RAGGED
    dy, x, wg, wu, g, u = exact_inputs(counts, KINDS, 200, 264, 0, after=0)
    off = offsets_of(counts)
    dx, dwg, dwu = sa.grouped_gated_linear_backward(dy, x, wg, wu, off, g, u, act="silu")
    assert torch.equal(sa.grouped_gated_linear_backward(dy, x, wg, wu, off, g, u, act="silu", with_dw=False)[0], dx)
    _, a, b = sa.grouped_gated_linear_backward(dy, x, wg, wu, off, g, u, act="silu", with_dx=False)
    assert torch.equal(a, dwg) and torch.equal(b, dwu)


# ---- real values -----------------------------------------------------------------

def real_inputs(counts, kinds, d_in, d_out, seed):
    r = np.random.default_rng(seed)
    T, n = sum(counts), len(counts)
    rows = lambda i: np.concatenate([np.full(c, 2.0**k[i]) for c, k in zip(counts, kinds)])[:, None]  # noqa: E731
    each = np.array([2.0**k[2] for k in kinds])[:, None, None]
    sizes = np.exp2(r.uniform(-2, 2, (T, 1))) * np.exp2(r.uniform(-2, 2, (1, d_out)))
    return (r.uniform(0.25, 1, (T, d_out)) * r.choice([-1, 1], (T, d_out)) * sizes * rows(0),
            r.standard_normal((T, d_in)) * rows(2), r.standard_normal((n, d_in, d_out)) * each,
            r.standard_normal((n, d_in, d_out)) * each, r.uniform(0.5, 2, (T, d_out)) * rows(1),
            r.uniform(0.5, 2, (T, d_out)) * rows(1))


@pytest.mark.parametrize("tile, split", [(-1, -1), (0, 8), (1, 64), (2, 64), (3, 0), (4, 256)])
@pytest.mark.parametrize("act", ["relu2", "silu", "gelu"])
def test_real_values(tuning, act, tile, split):  # noqa: F811
    """dx and dW of each expert within the dense layers' bounds of the definition
    on its rows alone."""
    tuning(tile, split)
    counts, kinds, d_in, d_out = [40, 0, 130, 33, 1, 65], [SMALL, SMALL, LARGE, PLAIN, LARGE, SMALL], 72, 264
    a = [dev(v) for v in real_inputs(counts, kinds, d_in, d_out, 9)]
    off = offsets_of(counts)
    dy, x, wg, wu, g, u = a
    dx, dwt, db = sa.grouped_linear_backward(dy, x, wg, off, act=act, pre=g, with_dbias=True)
    gx, dwg, dwu = sa.grouped_gated_linear_backward(dy, x, wg, wu, off, g, u, act=act)
    for e, r in by_expert(counts):
        DY, X, WG, WU, G, U = f64(dy[r]), f64(x[r]), f64(wg[e]), f64(wu[e]), f64(g[r]), f64(u[r])
        n = len(DY)
        d = DY * ol.slope(act, G)
        want = ol.linear_backward(DY, X, WG, act, G)
        representable(*want[:2])
        for axis, got, w, f in ((1, dx[r], want[0], lambda v: v @ np.abs(WG).T), (0, dwt[e], want[1], lambda v: np.abs(X).T @ v)):
            err = rounded(d, np.abs(DY), G, axis)
            close(got, w, f(err) + d.shape[axis] * E * f(np.abs(d) + err))
        if np.abs(d.sum(0)).max() < 30000:
            close(db[e], want[2], (np.abs(DY) * (np.abs(G) + 1) * 2.0**-18 + (n + 2) * E * np.abs(d)).sum(0))
        dg, du = DY * U * ol.slope(act, G), DY * ol.act(act, G)
        wdx, wdg, wdu = ol.gated_backward(DY, X, WG, WU, G, U, act)
        representable(wdx, wdg, wdu)
        both, W = np.concatenate([dg, du], 1), np.abs(np.concatenate([WG, WU], 1)).T
        scale = np.concatenate([np.abs(DY * U), np.abs(DY) * (np.abs(G) + 1)], 1)
        err = rounded(both, scale, np.concatenate([G, G], 1), 1)
        close(gx[r], wdx, err @ W + 2 * d_out * E * ((np.abs(both) + err) @ W))
        for got, w, v, s in ((dwg[e], wdg, dg, scale[:, :d_out]), (dwu[e], wdu, du, scale[:, d_out:])):
            err = rounded(v, s, G, 0)
            close(got, w, np.abs(X).T @ err + n * E * (np.abs(X).T @ (np.abs(v) + err)))
