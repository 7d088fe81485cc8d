"""Linear layers grouped by expert on the GPU against the fp64 definition.

With small integers every sum is exact in fp32 in any order, so outputs must
equal the correctly rounded definition bit for bit.  With real inputs the
bounds are the dense layers': half a step of the output's type, the fp32 sum's
error and the activation's."""

import numpy as np
import pytest
import torch

import sparse_input_gemv_amd as sa
from oracle import grouped as og
from oracle import linear as ol
from test_linear import DEV, E, TYPES, act_err, close, f64, half_step, ints, same
from test_linear import tuning  # noqa: F401

pytestmark = pytest.mark.gpu

# rows of each expert: none, one, several tiles of every height; one expert;
# all rows with one of many; more experts than a wave has lanes
COUNTS = {
    "ragged": [0, 1, 5, 0, 17, 64, 3, 0],
    "one": [37],
    "one of many": [0] * 11 + [131] + [0] * 9,
    "tiles": [300, 16, 257, 0, 128, 33],
    "64": [(3 * i) % 7 for i in range(64)],
    "65": [1] * 65,
    "200": [(i * i) % 5 for i in range(200)],
    "512": [i % 3 == 0 for i in range(512)],
    "none": [0, 0, 0],
}
DIMS = [(8, 8), (40, 72), (200, 264), (72, 1032)]


def offsets_of(counts, start=0):
    return torch.tensor(np.concatenate([[0], np.cumsum(counts)]) + start, dtype=torch.int32, device=DEV)


def by_expert(counts, start=0):
    o = offsets_of(counts, start).tolist()
    return [(e, slice(a, b)) for e, (a, b) in enumerate(zip(o, o[1:])) if b > a]


def relu64(z, act):
    p = z.clamp(min=0)
    return z if act == "none" else p if act == "relu" else p * p


def room(counts, before=2, after=3):
    return before + sum(map(int, counts)) + after


def kept(out, mark, counts, start):
    """Rows outside every expert's still hold the mark."""
    n = sum(map(int, counts))
    assert (out[:start] == mark).all() and (out[start + n:] == mark).all()


def nan_outside(x, counts, start):
    n = sum(map(int, counts))
    x[:start] = float("nan")
    x[start + n:] = float("nan")
    return x


@pytest.mark.parametrize("name", COUNTS)
@pytest.mark.parametrize("dtype", TYPES, ids=["fp16", "bf16"])
def test_forward_exact(name, dtype):
    counts, start = COUNTS[name], 2
    T, n = room(counts), len(counts)
    off = offsets_of(counts, start)
    for d_in, d_out in DIMS:
        x = nan_outside(ints((T, d_in), -2, 2, dtype, 1), counts, start)
        wt, wu = ints((n, d_in, d_out), -2, 2, dtype, 2), ints((n, d_in, d_out), -1, 1, dtype, 3)
        bias, res = ints((n, d_out), -9, 9, dtype, 4), ints((T, d_out), -50, 50, dtype, 5)
        y = sa.grouped_linear(x, wt, off, y=torch.full((T, d_out), 7, dtype=dtype, device=DEV))
        z, pre = (torch.full((T, d_out), 7, dtype=dtype, device=DEV) for _ in range(2))
        sa.grouped_linear(x, wt, off, bias=bias, act="relu2", residual=res, y=z, pre=pre)
        h, g, u, h2 = (torch.full((T, d_out), 7, dtype=dtype, device=DEV) for _ in range(4))
        sa.grouped_gated_linear(x, wt, wu, off, act="relu", h=h, g=g, u=u)
        sa.grouped_gated_linear(x, wt, wu, off, act="relu", h=h2)
        for out in (y, z, pre, h, g, u, h2):
            kept(out, 7, counts, start)
        for e, r in by_expert(counts, start):
            a, b = x[r].double() @ wt[e].double(), x[r].double() @ wu[e].double()
            same(y[r], a)
            same(pre[r], a + bias[e].double())
            same(z[r], relu64(a + bias[e].double(), "relu2") + res[r].double())
            same(g[r], a)
            same(u[r], b)
            same(h[r], a.clamp(min=0) * b)
            same(h2[r], a.clamp(min=0) * b)
        r0 = res.clone()  # in place on the residual
        sa.grouped_linear(x, wt, off, residual=r0, y=r0)
        for e, r in by_expert(counts, start):
            same(r0[r], x[r].double() @ wt[e].double() + res[r].double())


def check_backward(counts, start, d_in, d_out, dtype, acts=("none", "relu")):
    T, n = room(counts), len(counts)
    off = offsets_of(counts, start)
    x = nan_outside(ints((T, d_in), -2, 2, dtype, 11), counts, start)
    wt, wu = ints((n, d_in, d_out), -2, 2, dtype, 12), ints((n, d_in, d_out), -1, 1, dtype, 13)
    dy = nan_outside(ints((T, d_out), -1, 1, dtype, 14), counts, start)
    pre = nan_outside(ints((T, d_out), -3, 3, dtype, 15), counts, start)
    u = nan_outside(ints((T, d_out), -2, 2, dtype, 16), counts, start)
    for act in acts:
        dx = torch.full((T, d_in), 7, dtype=dtype, device=DEV)
        dwt = torch.full((n, d_in, d_out), float("nan"), dtype=dtype, device=DEV)
        _, _, db = sa.grouped_linear_backward(dy, x, wt, off, act=act, pre=pre, with_dbias=True, dx=dx, dwt=dwt)
        kept(dx, 7, counts, start)
        w64, b64 = torch.zeros(dwt.shape, dtype=torch.float64, device=DEV), torch.zeros(n, d_out, dtype=torch.float64, device=DEV)
        for e, r in by_expert(counts, start):
            p = pre[r].double().clamp(min=0)
            d = dy[r].double() * (1.0 if act == "none" else (p > 0).double())
            same(dx[r], d @ wt[e].double().T)
            w64[e], b64[e] = x[r].double().T @ d, d.sum(0)
        same(dwt, w64)
        same(db, b64)
    dx = torch.full((T, d_in), 7, dtype=dtype, device=DEV)
    _, dwg, dwu = sa.grouped_gated_linear_backward(dy, x, wt, wu, off, pre, u, act="relu", dx=dx)
    kept(dx, 7, counts, start)
    g64, u64 = torch.zeros(dwg.shape, dtype=torch.float64, device=DEV), torch.zeros(dwg.shape, dtype=torch.float64, device=DEV)
    for e, r in by_expert(counts, start):
        dg = dy[r].double() * u[r].double() * (pre[r] > 0).double()
        du = dy[r].double() * pre[r].double().clamp(min=0)
        same(dx[r], dg @ wt[e].double().T + du @ wu[e].double().T)
        g64[e], u64[e] = x[r].double().T @ dg, x[r].double().T @ du
    same(dwg, g64)
    same(dwu, u64)


@pytest.mark.parametrize("name", COUNTS)
@pytest.mark.parametrize("dtype", TYPES, ids=["fp16", "bf16"])
def test_backward_exact(name, dtype):
    for d_in, d_out in DIMS:
        check_backward(COUNTS[name], 2, d_in, d_out, dtype)


@pytest.mark.parametrize("split", [0, 8, 64, 512])
@pytest.mark.parametrize("tile", range(5))
def test_every_tile_and_split(tuning, tile, split):  # noqa: F811
    """All compiled tiles, whole and shared: shares that cross tiles and
    experts, more shares than steps, every epilogue, both gradients."""
    tuning(tile, split)
    for counts, d_in, d_out, dt in (([1], 200, 72, torch.float16), ([40, 0, 37, 90, 1, 300, 0, 2], 584, 392, torch.bfloat16),
                                    ([530, 3, 260], 328, 1032, torch.float16)):
        T, n, off = room(counts), len(counts), offsets_of(counts, 2)
        x = nan_outside(ints((T, d_in), -2, 2, dt, 90), counts, 2)
        wt, wu = ints((n, d_in, d_out), -2, 2, dt, 92), ints((n, d_in, d_out), -1, 1, dt, 93)
        bias, res = ints((n, d_out), -9, 9, dt, 94), ints((T, d_out), -50, 50, dt, 91)
        y = sa.grouped_linear(x, wt, off)
        z, pre = sa.grouped_linear(x, wt, off, bias=bias, act="relu", residual=res, with_pre=True)
        zr = sa.grouped_linear(x, wt, off, residual=res)
        h, g, u = sa.grouped_gated_linear(x, wt, wu, off, act="relu", with_gu=True)
        h2 = sa.grouped_gated_linear(x, wt, wu, off, act="relu")
        for e, r in by_expert(counts, 2):
            a, b = x[r].double() @ wt[e].double(), x[r].double() @ wu[e].double()
            same(y[r], a)
            same(zr[r], a + res[r].double())
            same(pre[r], a + bias[e].double())
            same(z[r], (a + bias[e].double()).clamp(min=0) + res[r].double())
            same(g[r], a)
            same(u[r], b)
            same(h[r], a.clamp(min=0) * b)
            same(h2[r], a.clamp(min=0) * b)
        check_backward(counts, 2, d_in, d_out, dt)


@pytest.mark.parametrize("counts, d_in, d_out", [([2, 0, 5, 1, 3, 0, 4, 1], 4096, 1424), ([700, 40, 260], 1032, 4168),
                                                 ([16] * 60 + [300, 0, 1, 40], 1024, 1032), ([1], 4096, 4096)], ids=str)
def test_layer_sizes_exact(counts, d_in, d_out):
    dtype = torch.bfloat16
    n, T, off = len(counts), sum(counts), offsets_of(counts)
    x = ints((T, d_in), -2, 2, dtype, 60)
    both = ints((n, d_in, 2 * d_out), -1, 1, dtype, 61)
    wg, wu = both[:, :, :d_out], both[:, :, d_out:]  # side by side
    dh, g = ints((T, d_out), -1, 1, dtype, 62), ints((T, d_out), -2, 2, dtype, 64)
    u = ints((T, d_out), -2, 2, dtype, 63)
    y, h = sa.grouped_linear(x, wg, off), sa.grouped_gated_linear(x, wg, wu, off, act="relu")
    out = torch.full((n, d_in, 2 * d_out), float("nan"), dtype=dtype, device=DEV)
    dx, dwg, dwu = sa.grouped_gated_linear_backward(dh, x, wg, wu, off, g, u, act="relu",
                                                    dwgt=out[:, :, :d_out], dwut=out[:, :, d_out:])
    assert torch.isfinite(out).all()
    for e, r in by_expert(counts):
        a, b = x[r].double() @ wg[e].double(), x[r].double() @ wu[e].double()
        same(y[r], a)
        same(h[r], a.clamp(min=0) * b)
        dg, du = dh[r].double() * u[r].double() * (g[r] > 0).double(), dh[r].double() * g[r].double().clamp(min=0)
        same(dx[r], dg @ wg[e].double().T + du @ wu[e].double().T)
        same(dwg[e], x[r].double().T @ dg)
        same(dwu[e], x[r].double().T @ du)


def test_strides():
    """Every matrix a window of a NaN matrix; experts' weights and gradients as
    column blocks of common rows; one weight for all experts."""
    dt, counts, d_in, d_out = torch.float16, [3, 0, 40, 21], 136, 72
    n, T, off = len(counts), sum(counts), offsets_of(counts)

    def window(v):
        w = torch.full((v.shape[0] + 2, v.shape[1] + 24), float("nan"), dtype=dt, device=DEV)
        w[1:-1, 8:8 + v.shape[1]] = v
        return w[1:-1, 8:8 + v.shape[1]]

    x, dy = window(ints((T, d_in), -2, 2, dt, 1)), window(ints((T, d_out), -1, 1, dt, 2))
    wide = ints((d_in, n * d_out), -2, 2, dt, 3)
    wt = wide.view(d_in, n, d_out).transpose(0, 1)  # [n][d_in][d_out], expert stride d_out
    y = window(torch.zeros(T, d_out, dtype=dt, device=DEV))
    dx = window(torch.zeros(T, d_in, dtype=dt, device=DEV))
    dwide = torch.full((d_in, n * d_out), float("nan"), dtype=dt, device=DEV)
    dwt = dwide.view(d_in, n, d_out).transpose(0, 1)
    sa.grouped_linear(x, wt, off, y=y)
    sa.grouped_linear_backward(dy, x, wt, off, dx=dx, dwt=dwt)
    shared = sa.grouped_linear(x, wt[2:3].expand(n, d_in, d_out), off)
    for e, r in by_expert(counts):
        same(y[r], x[r].double() @ wt[e].double())
        same(dx[r], dy[r].double() @ wt[e].double().T)
        same(dwt[e], x[r].double().T @ dy[r].double())
        same(shared[r], x[r].double() @ wt[2].double())
    assert (dwt[1] == 0).all()


@pytest.mark.parametrize("offsets", [[0, 30, 10, 50, 40, 64], [-5, 7, 7, 200, 3, 64], [64, 0, 0, 0, 0, 1 << 30],
                                     [9, 1, 2, -(1 << 31), 60, 61], [(1 << 31) - 1] * 6], ids=str)
def test_offsets_of_any_values(offsets):
    T, d_in, d_out, dt = 64, 72, 136, torch.bfloat16
    off = torch.tensor(offsets, dtype=torch.int32, device=DEV)
    clean = og.clean_offsets(offsets, T)
    x, dy = ints((T, d_in), -2, 2, dt, 1), ints((T, d_out), -1, 1, dt, 2)
    wt = ints((5, d_in, d_out), -2, 2, dt, 3)
    y = torch.full((T, d_out), 9, dtype=dt, device=DEV)
    dx = torch.full((T, d_in), 9, dtype=dt, device=DEV)
    sa.grouped_linear(x, wt, off, y=y)
    _, dwt, db = sa.grouped_linear_backward(dy, x, wt, off, dx=dx, with_dbias=True)
    for e, r in enumerate(og.parts(clean)):
        same(y[r], x[r].double() @ wt[e].double())
        same(dx[r], dy[r].double() @ wt[e].double().T)
        same(dwt[e], x[r].double().T @ dy[r].double())
        same(db[e], dy[r].double().sum(0))
    for out in (y, dx):
        assert (out[:clean[0]] == 9).all() and (out[clean[-1]:] == 9).all()


def test_offsets_past_32_bits():
    """Experts' matrices, and rows, whose last lie past 2^31 entries."""
    counts, d_in, d_out, dt = [20, 0, 70], 72, 136, torch.bfloat16
    t, step = sum(counts), 9 << 27
    o = offsets_of(counts)
    x, dy = ints((t, d_in), -2, 2, dt, 1), ints((t, d_out), -2, 2, dt, 2)
    wt = ints((len(counts), d_in, d_out), -2, 2, dt, 3)
    apart = lambda: torch.empty(2 * step + d_in * d_out, dtype=dt, device=DEV).as_strided(  # noqa: E731
        wt.shape, (step, d_out, 1))
    far = apart().copy_(wt)
    assert torch.equal(sa.grouped_linear(x, far, o), sa.grouped_linear(x, wt, o))
    assert torch.equal(sa.grouped_gated_linear(x, wt, far, o), sa.grouped_gated_linear(x, wt, wt, o))
    dx, dwt, _ = sa.grouped_linear_backward(dy, x, wt, o)
    fx, fwt, _ = sa.grouped_linear_backward(dy, x, far, o, dwt=apart())
    assert torch.equal(fx, dx) and torch.equal(fwt, dwt)
    del far, fwt

    counts, d_in, d_out = [70000, 1, 0, 70000], 8, 16384
    t, o = sum(counts), offsets_of(counts)
    x, wt = ints((t, d_in), -2, 2, dt, 4), ints((len(counts), d_in, d_out), -2, 2, dt, 5)
    y = sa.grouped_linear(x, wt, o)
    assert y.numel() > 2**31
    ends = [(0, slice(0, 300)), (1, slice(70000, 70001)), (3, slice(t - 300, t))]
    for e, r in ends:
        same(y[r], x[r].double() @ wt[e].double())
    y.clamp_(-1, 1)
    dx, dwt, db = sa.grouped_linear_backward(y, x, wt, o, with_dbias=True)
    for e, r in ends:
        same(dx[r], y[r].double() @ wt[e].double().T)
    for e, rows in by_expert(counts):
        parts = [slice(i, min(i + 20000, rows.stop)) for i in range(rows.start, rows.stop, 20000)]
        same(dwt[e], sum(x[r].double().T @ y[r].double() for r in parts))  # sums below 2^24
        same(db[e], sum(y[r].double().sum(0) for r in parts))


def test_empty():
    off = torch.zeros(4, dtype=torch.int32, device=DEV)
    x = torch.empty(0, 64, dtype=torch.float16, device=DEV)
    wt = ints((3, 64, 40), -2, 2, torch.float16, 1)
    assert sa.grouped_linear(x, wt, off).shape == (0, 40)
    assert sa.grouped_gated_linear(x, wt, wt, off).shape == (0, 40)
    nan = torch.full((3, 64, 40), float("nan"), dtype=torch.float16, device=DEV)
    dx, dwt, db = sa.grouped_linear_backward(x.new_empty(0, 40), x, wt, off, with_dbias=True, dwt=nan)
    assert dx.shape == (0, 64) and (dwt == 0).all() and (db == 0).all()


# ---- real values -----------------------------------------------------------------

@pytest.mark.parametrize("act", ["none", "silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("dtype", TYPES, ids=["fp16", "bf16"])
def test_real_values(dtype, act):
    rng = np.random.default_rng(5)
    counts, d_in, d_out = [70, 0, 1, 20, 300], 328, 136
    n, T, off = len(counts), sum(counts), offsets_of(counts)

    def dev(*shape, std=1.0):
        return torch.from_numpy(rng.standard_normal(shape) * std).to(dtype).to(DEV)

    x, wt, wu, bias = dev(T, d_in), dev(n, d_in, d_out, std=0.06), dev(n, d_in, d_out, std=0.06), dev(n, d_out)
    dy = dev(T, d_out, std=0.1)
    o = off.tolist()
    y, pre = sa.grouped_linear(x, wt, off, bias=bias, act=act, with_pre=True)
    wy, wpre = og.linear(f64(x), f64(wt), o, f64(bias), act)
    X, W, U, DY = f64(x), f64(wt), f64(wu), f64(dy)
    mag = og.linear(np.abs(X), np.abs(W), o, np.abs(f64(bias)))[1]
    err = d_in * E * mag
    close(pre, wpre, err)
    close(y, wy, act_err(wpre, err, act) + 2 * E * np.abs(wy))
    # gradients of the rounded pre-activation: d rounded to the type for the products
    P = f64(pre)
    dx, dwt, db = sa.grouped_linear_backward(dy, x, wt, off, act=act, pre=pre, with_dbias=True)
    wdx, wdw, wdb = og.linear_backward(DY, X, W, o, act, P)
    d = DY * ol.slope(act, P)
    e = np.abs(DY) * (np.abs(P) + 1) * 2.0**-18 if act != "none" else np.zeros_like(d)
    floor = 2.0**-17 if dtype == torch.float16 and act != "none" else 0.0
    for k, q in by_expert(counts):
        r = e[q] + half_step(dtype) * (np.abs(d[q]) + e[q]) * (act != "none")
        rx = r + floor * np.abs(d[q]).max(axis=1, keepdims=True)
        rw = r + floor * np.abs(d[q]).max(axis=0, keepdims=True)
        close(dx[q], wdx[q], (rx + d_out * E * np.abs(d[q])) @ np.abs(W[k]).T)
        close(dwt[k], wdw[k], np.abs(X[q]).T @ (rw + (q.stop - q.start) * E * np.abs(d[q])))
        close(db[k], wdb[k], (e[q] + 2 * (q.stop - q.start) * E * np.abs(d[q])).sum(0))
    if act != "none":
        h, g, u = sa.grouped_gated_linear(x, wt, wu, off, act=act, with_gu=True)
        wh, wg, wuu = og.gated(X, W, U, o, act)
        mg, mu = og.linear(np.abs(X), np.abs(W), o)[1], og.linear(np.abs(X), np.abs(U), o)[1]
        eg, eu = d_in * E * mg, d_in * E * mu
        close(g, wg, eg)
        close(u, wuu, eu)
        close(h, wh, act_err(wg, eg, act) * (np.abs(wuu) + eu) + np.abs(ol.act(act, wg)) * eu + 2 * E * np.abs(wh))


@pytest.mark.parametrize("size", [2.0**-12, 1.0, 2.0**7])
def test_fp16_gradients_by_expert_ranges(size):
    """One expert's d is far smaller or larger than the others': columns are
    scaled by their largest among the expert's own rows, so the bound holds
    with that one."""
    rng = np.random.default_rng(9)
    counts, d_in, d_out = [40, 33, 0, 65], 72, 136
    T, off = sum(counts), offsets_of(counts)
    F = torch.float16
    to = lambda v: torch.from_numpy(np.ascontiguousarray(v)).to(F).to(DEV)  # noqa: E731
    pre, x = rng.standard_normal((T, d_out)), rng.standard_normal((T, d_in))
    pre[:40] *= size
    if size < 1:
        x[:40] *= 256
    gx, gw = to(x), to(rng.standard_normal((4, d_in, d_out)) * 2.0**-3)
    gdy, gpre = to(rng.standard_normal((T, d_out)) * 2.0**-4), to(pre)
    dx, dwt, _ = sa.grouped_linear_backward(gdy, gx, gw, off, act="relu2", pre=gpre)
    for e, r in by_expert(counts):
        DY, X, W, P = (f64(v) for v in (gdy[r], gx[r], gw[e], gpre[r]))
        d = DY * ol.slope("relu2", P)
        own = (half_step(F) + 2 * E) * np.abs(d)
        wdx, wdw, _ = ol.linear_backward(DY, X, W, "relu2", P)
        close(dx[r], wdx, (own + 2.0**-17 * np.abs(d).max(axis=1, keepdims=True) + d_out * E * np.abs(d)) @ np.abs(W).T)
        close(dwt[e], wdw, np.abs(X).T @ (own + 2.0**-17 * np.abs(d).max(axis=0, keepdims=True) + len(d) * E * np.abs(d)))


def test_inf_and_nan_stay_with_their_rows():
    dt, counts, d_in, d_out = torch.bfloat16, [20, 9, 35], 136, 72
    off, T = offsets_of(counts), sum(counts)
    x, wt = ints((T, d_in), -2, 2, dt, 1), ints((3, d_in, d_out), -2, 2, dt, 2)
    clean = sa.grouped_linear(x, wt, off)
    x[19, 5], x[30, 7] = float("nan"), float("inf")  # the last of expert 0, one of expert 2
    y = sa.grouped_linear(x, wt, off)
    rows = torch.ones(T, dtype=torch.bool, device=DEV)
    rows[19] = rows[30] = False
    assert torch.equal(y[rows], clean[rows]) and torch.isnan(y[19]).all() and not torch.isfinite(y[30]).all()
    dy = ints((T, d_out), -1, 1, dt, 3)
    _, dwt, _ = sa.grouped_linear_backward(dy, x, wt, off)
    assert torch.isfinite(dwt[1]).all()  # between the two


# ---- calls at once, graphs -----------------------------------------------------------

def block(i, off):
    """A gated feed-forward block of experts, forward and backward."""
    x, wg, wu, wd, dy = i
    h, g, u = sa.grouped_gated_linear(x, wg, wu, off, with_gu=True)
    y = sa.grouped_linear(h, wd, off, residual=x)
    dh, dwd, _ = sa.grouped_linear_backward(dy, h, wd, off)
    dx, dwg, dwu = sa.grouped_gated_linear_backward(dh, x, wg, wu, off, g, u)
    return y, dwd, dx, dwg, dwu


def block_inputs(T, n, d, f, dt, seed):
    gen = torch.Generator().manual_seed(seed)

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, generator=gen) * std).to(dt).to(DEV)

    return (normal(T, d), normal(n, d, f, std=0.1), normal(n, d, f, std=0.1), normal(n, f, d, std=0.1), normal(T, d, std=0.1))


@pytest.mark.parametrize("dtype", TYPES, ids=["fp16", "bf16"])
def test_block_against_the_experts_alone(dtype):
    """The operators together: equal to the dense layers' block on each
    expert's rows, within twice their bounds' roundings."""
    counts = [0, 33, 5, 130]
    i, off = block_inputs(sum(counts), 4, 264, 136, dtype, 3), offsets_of(counts)
    y, dwd, dx, dwg, dwu = block(i, off)
    x, wg, wu, wd, dy = i
    # relative to the largest: six roundings of half a step lie on the way to dW
    tol = 12 * half_step(dtype)
    for e, r in by_expert(counts):
        h, g, u = sa.gated_linear(x[r], wg[e], wu[e], with_gu=True)
        ay = sa.dense_linear(h, wd[e], residual=x[r])
        dh, adwd, _ = sa.dense_linear_backward(dy[r], h, wd[e])
        adx, adwg, adwu = sa.gated_linear_backward(dh, x[r], wg[e], wu[e], g, u)
        for got, want in ((y[r], ay), (dwd[e], adwd), (dx[r], adx), (dwg[e], adwg), (dwu[e], adwu)):
            want = want.double()
            assert (got.double() - want).abs().max() <= tol * want.abs().max()
    assert (dwd[0] == 0).all() and (dwg[0] == 0).all() and (dwu[0] == 0).all()


def test_equal_calls_give_equal_bits_on_streams_at_once():
    counts = [3, 0, 20, 1, 40]
    sets = [block_inputs(64, 5, 1032, 520, torch.float16, s) for s in range(3)]
    off = offsets_of(counts)
    want = [block(i, off) for i in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(device=DEV) for _ in sets]
    got = [[] for _ in sets]
    for _ in range(4):
        for k, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[k].append(block(sets[k], off))
    torch.cuda.synchronize()
    for k, w in enumerate(want):
        for b in got[k]:
            for a, c in zip(b, w):
                assert torch.equal(a, c)


@pytest.mark.parametrize("counts", [[3, 0, 20, 1, 40], [300, 2, 0, 0, 210]], ids=str)
def test_a_captured_block_follows_its_offsets(counts):
    T = sum(counts)
    i, off = block_inputs(T, 5, 264, 520, torch.bfloat16, 4), offsets_of(counts)
    block(i, off)
    torch.cuda.synchronize()
    side = torch.cuda.Stream(device=DEV)
    with torch.cuda.stream(side):
        block(i, off)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        outs = block(i, off)
    for k in range(4):
        other = offsets_of(np.roll(counts, k))
        off.copy_(other)
        for o in outs:
            o.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, block(i, other)):
            assert torch.equal(a, b)


def test_warns_outside_autograd():
    x = ints((4, 64), -2, 2, torch.bfloat16, 1).requires_grad_()
    wt, off = ints((2, 64, 40), -2, 2, torch.bfloat16, 2), offsets_of([1, 3])
    with pytest.warns(UserWarning, match="grouped_linear_backward"):
        assert not sa.grouped_linear(x, wt, off).requires_grad
    with pytest.warns(UserWarning, match="grouped_gated_linear_backward"):
        sa.grouped_gated_linear(x, wt, wt, off)


def test_python_refusals():
    dt = torch.float16
    x, wt, off = ints((4, 64), -2, 2, dt, 1), ints((2, 64, 40), -2, 2, dt, 2), offsets_of([1, 3])
    for call in (lambda: sa.grouped_linear(x, wt, off.long()), lambda: sa.grouped_linear(x, wt, off.cpu()),
                 lambda: sa.grouped_linear(x, wt, off[:2]), lambda: sa.grouped_linear(x, wt, off[None]),
                 lambda: sa.grouped_linear(x, wt[0], off), lambda: sa.grouped_linear(x[:, :32], wt, off),
                 lambda: sa.grouped_linear(x, wt.bfloat16(), off), lambda: sa.grouped_linear(x, wt.transpose(1, 2), off),
                 lambda: sa.grouped_linear(x, wt, off, bias=x[0, :40]), lambda: sa.grouped_linear(x, wt, off, act="tanh"),
                 lambda: sa.grouped_linear(x[0], wt, off), lambda: sa.grouped_gated_linear(x[0], wt, wt, off),
                 lambda: sa.grouped_linear_backward(x[:, :40], x, wt, off, act="silu"),
                 lambda: sa.grouped_gated_linear(x, wt, wt[:1], off)):
        with pytest.raises(ValueError):
            call()
    dwt = torch.empty(1, 64, 40, dtype=dt, device=DEV).expand(2, 64, 40)
    with pytest.raises(sa.SparseActError, match="overlap"):
        sa.grouped_linear_backward(ints((4, 40), -1, 1, dt, 3), x, wt, off, dwt=dwt)
