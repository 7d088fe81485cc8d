"""Layers grouped by expert whose 256-row tiles fill a round of workgroups and
leave a rest that is shared: by the automatic plan, with ragged experts, every
epilogue.  Integer values, so outputs equal the definition bit for bit.

The device decides whether sharing pays; its rule is computed here too, so that
no case becomes one of whole tiles unnoticed."""

import pytest
import torch

import sparse_input_gemv_amd as sa
from test_grouped import by_expert, kept, nan_outside, offsets_of, room
from test_linear import DEV, TYPES, ints, same

pytestmark = pytest.mark.gpu
IDS = ["fp16", "bf16"]
CUS = 256


def shared(op, counts, d_in, d_out):
    """Asserts whole rounds of 256-row tiles and a rest that is shared, by the
    plan and by the device's rule: a step of a whole round takes 1.45 us, a
    share's partial sum 0.1, the reduction 4."""
    assert sa.grouped_plan(op, room(counts), len(counts), d_in, d_out) == {"tile_rows": 256, "split": CUS}
    n, k = (d_out, d_in) if op in ("forward", "gated") else (d_in, d_out)
    steps = -(-k // 64) * (2 if op == "gated_dx" else 1)
    tiles = sum(-(-c // 256) for c in counts) * -(-n // (128 if op == "gated" else 256))
    rest = tiles % CUS
    assert tiles > CUS and rest > 0
    assert (CUS - rest) * steps * 1.45 > 1.02 * CUS * ((CUS + rest) * 0.1 + 4)


def marked(*shape, dtype):
    return torch.full(shape, 7, dtype=dtype, device=DEV)


# tiles of several experts in the rest, one of a single row, experts without rows at
# both ends; an expert's rows end inside a tile, columns and the last step are odd
COUNTS = [0, 1300, 0, 700, 257, 1, 2300, 0]
FEW = [0, 700, 0, 1000, 257, 1, 300, 0]


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
def test_forward(dtype):
    counts, d_in, d_out, start = COUNTS, 2824, 3848, 2
    shared("forward", counts, d_in, d_out)
    T, n, off = room(counts), len(counts), offsets_of(counts, start)
    x = nan_outside(ints((T, d_in), -2, 2, dtype, 1), counts, start)
    wt, bias = ints((n, d_in, d_out), -2, 2, dtype, 2), ints((n, d_out), -9, 9, dtype, 3)
    res = ints((T, d_out), -50, 50, dtype, 4)
    y, b, r, z, pre = (marked(T, d_out, dtype=dtype) for _ in range(5))
    sa.grouped_linear(x, wt, off, y=y)
    sa.grouped_linear(x, wt, off, bias=bias, y=b)
    sa.grouped_linear(x, wt, off, residual=res, y=r)
    sa.grouped_linear(x, wt, off, bias=bias, act="relu", residual=res, y=z, pre=pre)
    for out in (y, b, r, z, pre):
        kept(out, 7, counts, start)
    for e, q in by_expert(counts, start):
        a = x[q].double() @ wt[e].double()
        ab = a + bias[e].double()
        same(y[q], a)
        same(b[q], ab)
        same(r[q], a + res[q].double())
        same(pre[q], ab)
        same(z[q], ab.clamp(min=0) + res[q].double())


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
def test_gated_forward(dtype):
    counts, d_in, d_out, start = FEW, 2824, 3336, 2
    shared("gated", counts, d_in, d_out)
    T, n, off = room(counts), len(counts), offsets_of(counts, start)
    x = nan_outside(ints((T, d_in), -1, 1, dtype, 1), counts, start)
    wg, wu = ints((n, d_in, d_out), -2, 2, dtype, 2), ints((n, d_in, d_out), -1, 1, dtype, 3)
    h, h2, g, u = (marked(T, d_out, dtype=dtype) for _ in range(4))
    sa.grouped_gated_linear(x, wg, wu, off, act="relu", h=h)
    sa.grouped_gated_linear(x, wg, wu, off, act="relu", h=h2, g=g, u=u)
    for out in (h, h2, g, u):
        kept(out, 7, counts, start)
    assert torch.equal(h, h2)
    for e, q in by_expert(counts, start):
        a, b = x[q].double() @ wg[e].double(), x[q].double() @ wu[e].double()
        same(g[q], a)
        same(u[q], b)
        same(h[q], a.clamp(min=0) * b)


@pytest.mark.parametrize("act", ["none", "relu"])
@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
def test_dx(dtype, act):
    counts, d_in, d_out, start = COUNTS, 3848, 2824, 2
    shared("dx", counts, d_in, d_out)
    T, n, off = room(counts), len(counts), offsets_of(counts, start)
    x, wt = ints((T, d_in), -2, 2, dtype, 1), ints((n, d_in, d_out), -2, 2, dtype, 2)
    dy, pre = (nan_outside(ints((T, d_out), -2, 2, dtype, s), counts, start) for s in (3, 4))
    dx = marked(T, d_in, dtype=dtype)
    sa.grouped_linear_backward(dy, x, wt, off, act=act, pre=pre, dx=dx, with_dwt=False)
    kept(dx, 7, counts, start)
    for e, q in by_expert(counts, start):
        same(dx[q], (dy[q].double() * (1.0 if act == "none" else (pre[q] > 0).double())) @ wt[e].double().T)


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
def test_gated_dx(dtype):
    counts, d_in, d_out, start = COUNTS, 3848, 1416, 2
    shared("gated_dx", counts, d_in, d_out)
    T, n, off = room(counts), len(counts), offsets_of(counts, start)
    x, wg, wu = (ints(s, -2, 2, dtype, k) for k, s in enumerate(((T, d_in), (n, d_in, d_out), (n, d_in, d_out))))
    dh, g, u = (nan_outside(ints((T, d_out), -2, 2, dtype, s), counts, start) for s in (3, 4, 5))
    dx = marked(T, d_in, dtype=dtype)
    sa.grouped_gated_linear_backward(dh, x, wg, wu, off, g, u, act="relu", dx=dx, with_dw=False)
    kept(dx, 7, counts, start)
    for e, q in by_expert(counts, start):
        dg, du = dh[q].double() * u[q].double() * (g[q] > 0).double(), dh[q].double() * g[q].double().clamp(min=0)
        same(dx[q], dg @ wg[e].double().T + du @ wu[e].double().T)


def test_equal_calls_and_replays_give_equal_bits():
    """Real values: the rest's sums are in the offsets' order whatever runs beside."""
    counts, d_in, d_out, dt = COUNTS, 2824, 3848, torch.bfloat16
    T, n, off = room(counts), len(counts), offsets_of(counts, 2)
    gen = torch.Generator(device=DEV).manual_seed(1)
    x = torch.randn(T, d_in, generator=gen, device=DEV).to(dt)
    wt = torch.randn(n, d_in, d_out, generator=gen, device=DEV).to(dt)
    y = marked(T, d_out, dtype=dt)
    want = sa.grouped_linear(x, wt, off, act="silu", y=y.clone())
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream(device=DEV)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        sa.grouped_linear(x, wt, off, act="silu", y=y)
    for _ in range(3):
        y.fill_(7)
        assert torch.equal(sa.grouped_linear(x, wt, off, act="silu", y=marked(T, d_out, dtype=dt)), want)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want)
    # another split of the rows: the tiles, the rest and its shares are found anew
    other = offsets_of(COUNTS[::-1], 2)
    off.copy_(other)
    y.fill_(7)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, sa.grouped_linear(x, wt, other, act="silu", y=marked(T, d_out, dtype=dt)))
