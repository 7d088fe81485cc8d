"""The fp16 gradients of the dense linear layers over fp16's range: products d
of the incoming gradient and the slope that lie above fp16's largest value, in
its subnormals or below them, while dx and dW are ordinary numbers.

The bound: a d is off by half a step of itself, its evaluation's error, and
2^-17 of the largest of its row (for dx; gated: of dg and du together) or of
its column (for dW): half a subnormal step, 2^-25, of values whose largest is
2^-8 at least, unscaled or by a power of two."""

import numpy as np
import pytest
import torch

import sparse_input_gemv_amd as sa
from oracle import linear as ol
from test_linear import DEV, E, f64, half_step, tuning  # noqa: F401
from test_linear import close as close_where_ordered

pytestmark = pytest.mark.gpu

F16 = torch.float16
H = half_step(F16)
MAX = 65504.0
# one row to several tiles: shares, dx and dW in one launch, whole tiles; odd sizes
SHAPES = [(1, 8, 8), (2, 40, 1032), (37, 136, 200), (300, 1024, 1032), (515, 264, 520), (2100, 72, 40)]


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(F16).to(DEV)


def rounded(d, scale, z, axis):
    """Error of d as the products read it: slopes are good to 2^-18 (of values
    up to |z| + 1), then half a step and the floor of its row or column."""
    e = scale * (np.abs(z) + 1) * 2.0**-18 + 2 * E * np.abs(d)
    return e + H * (np.abs(d) + e) + 2.0**-17 * np.abs(d).max(axis=axis, keepdims=True)


def close(got, want, err):
    assert torch.isfinite(got).all()  # no comparison with a NaN is false here
    close_where_ordered(got, want, err)


def representable(*arrays):
    for a in arrays:
        assert np.abs(a).max() < MAX / 2
        assert np.abs(a).max() > 2.0**-18  # not all rounded to nothing


def check_linear(dy, x, wt, z, act):
    dx, dwt, db = sa.dense_linear_backward(dev(dy), dev(x), dev(wt), act=act, pre=dev(z), with_dbias=True)
    DY, X, W, Z = (f64(dev(a)) for a in (dy, x, wt, z))
    d = DY * ol.slope(act, Z)
    wdx, wdw, _ = ol.linear_backward(DY, X, W, act, Z)
    representable(wdx, wdw)
    for axis, got, want, f in ((1, dx, wdx, lambda v: v @ np.abs(W).T), (0, dwt, wdw, lambda v: np.abs(X).T @ v)):
        e = rounded(d, np.abs(DY), Z, axis)
        n = d.shape[axis]
        close(got, want, f(e) + n * E * f(np.abs(d) + e))
    if np.abs(d.sum(0)).max() < MAX / 2:
        close(db, d.sum(0), (np.abs(DY) * (np.abs(Z) + 1) * 2.0**-18 + (len(d) + 2) * E * np.abs(d)).sum(0))
    return d


def check_gated(dh, x, wg, wu, g, u, act):
    dx, dwg, dwu = sa.gated_linear_backward(dev(dh), dev(x), dev(wg), dev(wu), dev(g), dev(u), act=act)
    DH, X, WG, WU, G, U = (f64(dev(a)) for a in (dh, x, wg, wu, g, u))
    dg, du = DH * U * ol.slope(act, G), DH * ol.act(act, G)
    wdx, wdg, wdu = ol.gated_backward(DH, X, WG, WU, G, U, act)
    representable(wdx, wdg, wdu)
    both = np.concatenate([dg, du], 1)
    scale = np.concatenate([np.abs(DH * U), np.abs(DH) * (np.abs(G) + 1)], 1)  # relu2's value: |g| |g|
    zz = np.concatenate([G, G], 1)
    W = np.abs(np.concatenate([WG, WU], 1)).T
    e = rounded(both, scale, zz, 1)
    close(dx, wdx, e @ W + 2 * dg.shape[1] * E * ((np.abs(both) + e) @ W))
    n = dg.shape[1]
    for got, want, d, s in ((dwg, wdg, dg, scale[:, :n]), (dwu, wdu, du, scale[:, n:])):
        e = rounded(d, s, G, 0)
        close(got, want, np.abs(X).T @ e + len(d) * E * (np.abs(X).T @ (np.abs(d) + e)))
    return dg, du


@pytest.mark.parametrize("act", ["relu2", "silu"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_large_d(shape, act):
    """|d| far above 65504 everywhere; small x and weights."""
    t, d_in, d_out = shape
    r = np.random.default_rng(1)
    x = 1e-3 / np.sqrt(t) * r.standard_normal((t, d_in))
    wt = 5e-4 / np.sqrt(d_out) * r.standard_normal((d_in, d_out))
    dy = np.sign(r.standard_normal((t, d_out))) * r.uniform(2e4, 6e4, (t, d_out))
    z = np.abs(r.standard_normal((t, d_out))) + 2
    d = check_linear(dy, x, wt, z, act)
    assert np.abs(d).max() > (MAX if act == "relu2" else MAX / 4)
    u = r.uniform(12, 36, (t, d_out))
    dg, du = check_gated(dy, x, wt, wt[::-1], z, u, act)
    assert np.abs(dg).max() > MAX and np.abs(du).max() > MAX


@pytest.mark.parametrize("act", ["relu", "gelu"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_small_d(shape, act):
    """|d| near and below fp16's smallest subnormal (6e-8); large x and weights."""
    t, d_in, d_out = shape
    r = np.random.default_rng(2)
    x, wt = 400 * r.uniform(1, 2, (t, d_in)), 400 * r.uniform(1, 2, (d_in, d_out))
    dy = r.uniform(2e-6, 4e-6, (t, d_out))
    z = r.uniform(0.5, 1.5, (t, d_out))
    check_linear(dy, x, wt, z, act)
    u = r.uniform(1e-3, 2e-3, (t, d_out))
    dg, _ = check_gated(dy, x, wt, wt, z, u, act)
    assert np.abs(dg).max() < 2.0**-24


@pytest.mark.parametrize("t", [5, 130, 300])
def test_one_entry_above_the_range(t):
    """A single d of 163840 among ordinary ones: every entry stays finite, and
    rows and columns without it keep the bits they have without it."""
    r = np.random.default_rng(3)
    d_in, d_out = 136, 1032
    x, wg, wu = r.standard_normal((t, d_in)), 0.02 * r.standard_normal((d_in, d_out)), 0.02 * r.standard_normal((d_in, d_out))
    dh, g, u = (r.standard_normal((t, d_out)) for _ in range(3))
    x[3] *= 0.05
    before = sa.gated_linear_backward(*(dev(a) for a in (dh, x, wg, wu, g, u)), act="relu2")
    dh[3, 700], u[3, 700], g[3, 700] = 64, 64, 20
    check_gated(dh, x, wg, wu, g, u, "relu2")
    after = sa.gated_linear_backward(*(dev(a) for a in (dh, x, wg, wu, g, u)), act="relu2")
    rows, cols = np.arange(t) != 3, np.arange(d_out) != 700
    # elsewhere only subnormal d are rounded more finely
    b, a = f64(before[0])[rows], f64(after[0])[rows]
    assert np.abs(a - b).max() <= 2 * H * np.abs(b).max()
    for k in (1, 2):
        b, a = f64(before[k])[:, cols], f64(after[k])[:, cols]
        assert np.abs(a - b).max() <= 2 * H * np.abs(b).max()


@pytest.mark.parametrize("t", [40, 300, 1100])
def test_rows_and_columns_of_every_size(t):
    """Rows of d from 2^-40 to 2^30 beside each other reach their rows of dx
    (fp16 holds the result through the weights' size), and columns as far
    apart their columns of dW."""
    r = np.random.default_rng(4)
    d_in, d_out = 136, 264
    z = np.abs(r.standard_normal((t, d_out))) + 0.1
    for axis in (0, 1):
        n = t if axis == 0 else d_out
        e = r.permutation(np.linspace(-20, 14, n))
        s = np.exp2(e)[:, None] if axis == 0 else np.exp2(e)[None]
        dh, u = s * r.uniform(0.5, 1, (t, d_out)), s * r.uniform(0.5, 1, (t, d_out))
        x, w = 2.0**-14 * r.uniform(0.5, 1, (t, d_in)), 2.0**-16 * r.uniform(0.5, 1, (d_in, d_out))
        DH, X, W, G, U = (f64(dev(a)) for a in (dh, x, w, z, u))
        dg, du = DH * U, DH * G
        dx, dwg, dwu = sa.gated_linear_backward(*(dev(a) for a in (dh, x, w, w, z, u)), act="relu")
        assert np.abs(dg).max() > 2.0**26 and np.abs(dg).min() < 2.0**-38
        if axis == 0:
            want = (dg + du) @ W.T
            fits = np.abs(want).max(1) < MAX / 2
            assert 0.5 < fits.mean()
            both = np.concatenate([dg, du], 1)
            e = (2 * E + H) * np.abs(both) + 2.0**-17 * np.abs(both).max(1, keepdims=True)
            WW = np.concatenate([W, W], 1).T
            close(dx[torch.from_numpy(fits).to(DEV)], want[fits],
                  (e @ WW + 4 * d_out * E * (np.abs(both) @ WW))[fits])
        else:
            for got, d in ((dwg, dg), (dwu, du)):
                want = X.T @ d
                fits = np.abs(want).max(0) < MAX / 2
                assert 0.5 < fits.mean()
                e = (2 * E + H) * np.abs(d) + 2.0**-17 * np.abs(d).max(0, keepdims=True)
                close(got[:, torch.from_numpy(fits).to(DEV)], want[:, fits],
                      (X.T @ e + 2 * t * E * (X.T @ np.abs(d)))[:, fits])


@pytest.mark.parametrize("split", [0, 64])
@pytest.mark.parametrize("tile", [0, 1, 2, 3, 4, 5])
def test_every_tile(tuning, tile, split):  # noqa: F811
    """Large and small d through every compiled tile, whole and shared, and
    with one of the two gradients alone."""
    tuning(tile, split)
    r = np.random.default_rng(5)
    for t, d_in, d_out in ((77, 200, 392), (300, 328, 264)):
        x, wt = r.standard_normal((t, d_in)), r.standard_normal((d_in, d_out))
        g, u, dh = (r.uniform(0.5, 2, (t, d_out)) for _ in range(3))
        for s in (2.0**-20, 2.0**13):
            k = 2.0**-4 if s < 1 else 2.0**-17
            ws = 1 / (k * 64) if s < 1 else 2.0**-13
            a = [dh * s, x * ws, wt * ws, wt * ws, g, u * 8]
            check_gated(*a, "relu2")
            check_linear(dh * s, x * ws, wt * ws, g * 8, "relu2")
            d = [dev(v) for v in a]
            full = sa.gated_linear_backward(*d, act="relu2")
            dx = sa.gated_linear_backward(*d, act="relu2", with_dw=False)[0]
            _, dwg, dwu = sa.gated_linear_backward(*d, act="relu2", with_dx=False)
            for p, q in zip(full, (dx, dwg, dwu)):
                assert torch.equal(p, q)


def test_non_finite_gradients_stay_in_their_row_and_column():
    """Inf and NaN in dy reach their row of dx and their column of dW only,
    small d beside them keep their size."""
    r = np.random.default_rng(6)
    t, d_in, d_out = 150, 136, 200
    x, wt = 100 * r.uniform(1, 2, (t, d_in)), 100 * r.uniform(1, 2, (d_in, d_out))
    dy, z = r.uniform(1e-6, 2e-6, (t, d_out)), r.uniform(0.1, 0.2, (t, d_out))
    dy[7, 11], dy[9, 60] = np.inf, np.nan
    dx, dwt, db = (f64(v) for v in sa.dense_linear_backward(dev(dy), dev(x), dev(wt), act="relu2", pre=dev(z),
                                                            with_dbias=True))
    rows, cols = np.isin(np.arange(t), (7, 9)), np.isin(np.arange(d_out), (11, 60))
    assert not np.isfinite(dx[rows]).any() and not np.isfinite(dwt[:, cols]).any()
    assert not np.isfinite(db[cols]).any()
    DY, X, W, Z = (f64(dev(a)) for a in (dy, x, wt, z))
    d = DY * 2 * Z
    for got, want in ((dx[~rows], d[~rows] @ W.T), (dwt[:, ~cols], X.T @ d[:, ~cols])):
        # half steps of d and of the result, 2^-17 of the largest; every term is positive
        assert np.abs(got - want).max() <= (2 * H + 2.0**-15) * want.max() + 2.0**-25


def test_graph_replays_with_other_ranges():
    """One captured call replayed with inputs of ordinary, large and small d
    in turn gives each the bits of its own eager call."""
    r = np.random.default_rng(7)
    t, d_in, d_out = 130, 136, 264
    base = [dev(v) for v in (r.uniform(0.5, 1, (t, d_out)), 2.0**-9 * r.standard_normal((t, d_in)),
                             2.0**-9 * r.standard_normal((d_in, d_out)), r.uniform(1, 2, (t, d_out)),
                             r.uniform(1, 2, (t, d_out)))]
    dh, x, w, g, u = (v.clone() for v in base)
    f = lambda: (*sa.gated_linear_backward(dh, x, w, w, g, u, act="relu2"),  # noqa: E731
                 *sa.dense_linear_backward(dh, x, w, act="relu2", pre=g, with_dbias=True))
    f()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = f()
    for k in (0, 15, 0, -18, -18, 0, 15):
        dh.copy_(base[0] * 2.0**k)
        want = [v.clone() for v in f()]
        for v in out:
            v.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, want):
            assert torch.equal(a, b)
        assert all(v.any() for v in want)
