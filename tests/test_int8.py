"""Linear layers in 8-bit integers on the GPU: codes and scales against the
fp64 oracle bit for bit, products against it within half a step of the output's
type and the epilogue's few fp32 roundings (the integer sums are exact)."""

import numpy as np
import pytest
import torch

import sparse_input_gemv_amd as sa
from oracle import int8 as oi
from oracle import linear as ol
from test_linear import DEV, E, TYPES, act_err, close, f64, ints
from test_linear import tuning  # noqa: F401

pytestmark = pytest.mark.gpu
IDS = ["fp16", "bf16"]


def rows_of(shape, dtype, seed, std=1.0):
    gen = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=gen) * std).to(dtype).to(DEV)


def same_codes(x, q, s):
    wq, ws = oi.quantize(f64(x))
    assert np.array_equal(s.cpu().numpy(), ws, equal_nan=True)
    got = q.cpu().numpy()
    assert np.array_equal(got, wq), f"{int((got != wq).sum())} of {wq.size} codes differ"


# a row per wave and per workgroup, every number of chunks per thread, rows read twice
@pytest.mark.parametrize("shape", [(1, 16), (3, 48), (1030, 16), (1025, 2048), (2, 2048), (5, 2064), (7, 4096), (3, 4112),
                                   (4, 8192), (3, 11008), (2, 16384), (2, 16400), (3, 131072)], ids=str)
@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
def test_tokens(shape, dtype):
    x = rows_of(shape, dtype, 3)
    x[0, 1:] *= 0.01  # one large value
    same_codes(x, *sa.act_quantize_int8(x))


@pytest.mark.parametrize("shape", [(16, 8), (48, 40), (256, 64), (272, 72), (1040, 520), (2064, 1032), (11008, 264),
                                   (131072, 8)], ids=str)
@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
def test_channels(shape, dtype):
    wt = rows_of(shape, dtype, 4, 0.02)
    wt[:, 0] = 0
    wq, sw = sa.weight_quantize_int8(wt)
    assert wq.shape == (shape[1], shape[0])
    same_codes(wt.T, wq, sw)


def every_value(dtype):
    """All finite values of a 16-bit type, a row of 2^15 of them with each of
    several largest magnitudes that cut the row off."""
    bits = torch.arange(1 << 16, dtype=torch.int32).to(torch.int16)
    v = bits.view(dtype)
    return v[torch.isfinite(v)]


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
def test_every_value_under_many_scales(dtype):
    v = every_value(dtype)
    mags = v.double().abs().unique()
    mags = mags[mags > 0]
    at = torch.linspace(0, len(mags) - 1, 160).long()
    d = 65536
    x = torch.zeros(len(at), d, dtype=dtype)
    for i, k in enumerate(at):
        keep = v[v.double().abs() <= mags[k]]
        x[i, :len(keep)] = keep
    x = x.to(DEV)
    same_codes(x, *sa.act_quantize_int8(x))


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
def test_halves_go_to_even(dtype):
    # the largest is 127 * 2^k: s = 2^k, and (j + 1/2) 2^k lies half way
    j = torch.arange(-64, 64, dtype=torch.float64)
    x = torch.zeros(3, 144, dtype=torch.float64)
    for r, k in enumerate((-7, 0, 3)):
        x[r, :128] = (j + 0.5) * 2.0**k
        x[r, 128] = 127 * 2.0**k
    x = x.to(dtype).to(DEV)
    q, s = sa.act_quantize_int8(x)
    assert s.tolist() == [2.0**-7, 1.0, 8.0]
    want = (2 * torch.round((j + 0.5) / 2)).to(torch.int8)  # the even neighbour
    assert torch.equal(q[:, :128].cpu(), want.expand(3, 128)) and (q[:, 128] == 127).all()
    same_codes(x, q, s)


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
def test_rows_without_a_scale(dtype):
    x = rows_of((6, 64), dtype, 5)
    x[0] = 0
    x[1] = -0.0
    x[2, 7], x[3, 9], x[4, 63] = float("inf"), float("nan"), float("-inf")
    q, s = sa.act_quantize_int8(x)
    assert (s[:2] == 0).all() and torch.isnan(s[2:5]).all() and (q[:5] == 0).all()
    same_codes(x[5:], q[5:], s[5:])
    wt = x.T.contiguous()  # [64][6] -> pad to 8 channels
    wt = torch.cat([wt, wt[:, :2]], dim=1).contiguous()
    wq, sw = sa.weight_quantize_int8(wt)
    same_codes(wt.T, wq, sw)
    # such a token's outputs are NaN, and no other's
    y = sa.int8_linear(x, *sa.weight_quantize_int8(rows_of((64, 40), dtype, 6)))
    assert torch.isnan(y[2:5]).all() and torch.isfinite(y[[0, 1, 5]]).all() and (y[:2] == 0).all()


def test_smallest_bf16_scales():
    x = torch.tensor([2.0**-133, -(2.0**-133), 0.0, 3 * 2.0**-133] * 4, dtype=torch.float64)
    x = torch.stack([x, x * 5, x * 2.0**20, x * 2.0**40]).to(torch.bfloat16).to(DEV)
    same_codes(x, *sa.act_quantize_int8(x))


def test_strided_quantisers():
    x = rows_of((20, 112), torch.float16, 7)[:, 8:88]
    q = torch.full((20, 112), 99, dtype=torch.int8, device=DEV)
    s = torch.empty(20, device=DEV)
    got, gs = sa.act_quantize_int8(x, xq=q[:, 16:96], sx=s)
    assert gs is s and (q[:, :16] == 99).all() and (q[:, 96:] == 99).all()
    same_codes(x, got, s)
    wt = rows_of((80, 96), torch.bfloat16, 8)[:, 16:88]
    q = torch.full((72, 112), 99, dtype=torch.int8, device=DEV)
    got, gs = sa.weight_quantize_int8(wt, wq=q[:, 16:96])
    assert (q[:, :16] == 99).all() and (q[:, 96:] == 99).all()
    same_codes(wt.T, got, gs)


# ---- products --------------------------------------------------------------------------

def codes(shape, seed):
    gen = torch.Generator().manual_seed(seed)
    return torch.randint(-127, 128, shape, generator=gen, dtype=torch.int8).to(DEV)


def scales(n, seed, about=2.0**-9):
    gen = torch.Generator().manual_seed(seed)
    return ((1 + torch.rand(n, generator=gen)) * about).to(DEV)


def check(x, sx, wq, sw, dtype, bias=None, act="none", res=None, **kw):
    y = sa.int8_linear(x, wq, sw, sx=sx, bias=bias, act=act, residual=res, dtype=dtype, **kw)
    xq, s = (x, sx) if sx is not None else sa.act_quantize_int8(x)
    want, z = oi.linear(xq.cpu().numpy(), s.cpu().numpy(), wq.cpu().numpy(), sw.cpu().numpy(),
                        None if bias is None else f64(bias), act, None if res is None else f64(res))
    prod = np.abs(z - (0 if bias is None else f64(bias)))
    ez = 2 * E * prod + E * np.abs(z)  # the sum's rounding to fp32 and two scales, then the bias
    close(y, want, act_err(z, ez, act) + 2 * E * (np.abs(z) + np.abs(want)))
    return y


ROWS = [1, 2, 3, 4, 5, 8, 9, 17, 33, 65, 129, 300]
DIMS = [(16, 8), (48, 40), (272, 136), (1040, 520), (4112, 264)]


@pytest.mark.parametrize("dims", DIMS, ids=str)
@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
def test_products(dims, dtype):
    d_in, d_out = dims
    wq, sw = codes((d_out, d_in), 1), scales(d_out, 2)
    bias = rows_of((d_out,), dtype, 3)
    for k, t in enumerate(ROWS):
        x, sx, res = codes((t, d_in), 10 + t), scales(t, t, 2.0**-7), rows_of((t, d_out), dtype, 5)
        check(x, sx, wq, sw, dtype)
        act = ("silu", "gelu", "relu2", "gelu_tanh", "relu")[k % 5]
        check(x, sx, wq, sw, dtype, bias=bias, act=act, res=res)
        xf = rows_of((t, d_in), dtype, 20 + t)
        y = check(xf, None, wq, sw, dtype, bias=bias, res=res)
        q, s = sa.act_quantize_int8(xf)  # quantised within the call or before it: the same bits
        assert torch.equal(y, sa.int8_linear(q, wq, sw, sx=s, bias=bias, residual=res, dtype=dtype))
        sa.int8_linear(xf, wq, sw, bias=bias, residual=res, y=res)  # in place on the residual
        assert torch.equal(res, y)


@pytest.mark.parametrize("t", [1, 2, 8, 40, 700])
def test_extreme_sums_are_exact(t):
    """Sums of 2^31 nearly, and differences of huge parts: products of codes
    whose sum fp32 could not hold; a scale of one shows the integer."""
    d_in, d_out = 131072, 16
    x = torch.full((t, d_in), 127, dtype=torch.int8, device=DEV)
    wq = torch.full((d_out, d_in), 127, dtype=torch.int8, device=DEV)
    wq[1] = -127
    wq[2, ::2] = -127
    wq[3, ::2] = -127
    wq[3, 1] = 126  # 0 - 127
    one = torch.ones(t, device=DEV), torch.ones(d_out, device=DEV)
    y = sa.int8_linear(x, wq, one[1] * 2.0**-16, sx=one[0], dtype=torch.float16).double()
    full = 127 * 127 * d_in / 65536
    assert (y[:, 0] == torch.tensor(full).half().double()).all() and (y[:, 1] == -y[:, 0]).all()
    assert (y[:, 2] == 0).all()
    y = sa.int8_linear(x, wq, one[1], sx=one[0], dtype=torch.float16).double()
    assert (y[:, 3] == -127).all() and torch.isinf(y[:, 0]).all()


@pytest.mark.parametrize("split", [0, 8, 64, 512])
@pytest.mark.parametrize("tile", range(6))
def test_every_tile_and_split(tuning, tile, split):  # noqa: F811
    tuning(tile, split)
    for t, d_in, d_out, dt in ((9, 208, 72, torch.float16), (77, 592, 392, torch.bfloat16), (530, 336, 1032, torch.float16),
                               (300, 80, 5128, torch.bfloat16)):
        x, sx = codes((t, d_in), 31), scales(t, 32, 2.0**-7)
        wq, sw = codes((d_out, d_in), 33), scales(d_out, 34)
        check(x, sx, wq, sw, dt)
        check(x, sx, wq, sw, dt, bias=rows_of((d_out,), dt, 35), act="silu", res=rows_of((t, d_out), dt, 36))


@pytest.mark.parametrize("shape", [(1, 4096, 11008), (8, 8192, 4096), (33, 11008, 4096), (1, 14336, 1024), (1, 65536, 72),
                                   (1, 65552, 72), (2048, 4096, 1424), (1, 16, 40008),
                                   # either side of where one kernel takes over from another
                                   (4, 16384, 264), (4, 16400, 264), (5, 4096, 11776), (5, 4096, 11768), (8, 8192, 5896),
                                   (8, 8208, 5896), (64, 4096, 4704), (64, 4096, 4712), (17, 11008, 2920),
                                   (17, 11008, 2928)], ids=str)
def test_layer_sizes(shape):
    t, d_in, d_out = shape
    dt = torch.bfloat16
    wq, sw = codes((d_out, d_in), 41), scales(d_out, 42)
    x = rows_of((t, d_in), dt, 43)
    y = sa.int8_linear(x, wq, sw)
    q, s = sa.act_quantize_int8(x)
    total = q.double() @ wq.double().T  # exact in fp64
    want = (total * sw.double()[None] * s.double()[:, None]).cpu().numpy()
    close(y, want, 3 * E * np.abs(want))


def test_strides():
    dt, d_in, d_out = torch.float16, 80, 72
    for t in (1, 5, 40):
        x = codes((t, 112), 1)[:, 16:96]
        wq = codes((d_out, 128), 2)[:, 32:112]
        sx, sw = scales(t, 3), scales(d_out, 4)
        y = torch.full((t + 2, d_out + 24), float("nan"), dtype=dt, device=DEV)
        res = torch.full((t, d_out + 24), float("nan"), dtype=dt, device=DEV)
        res[:, 8:80] = rows_of((t, d_out), dt, 5)
        check(x, sx, wq, sw, dt, res=res[:, 8:80], y=y[1:-1, 8:80])
        assert torch.isnan(y[:, :8]).all() and torch.isnan(y[:, 80:]).all() and torch.isnan(y[[0, -1]]).all()
        xf = rows_of((t, 104), dt, 6)[:, 8:88]
        check(xf, None, wq, sw, dt)


@pytest.mark.parametrize("t", [2, 9, 90])
def test_rows_of_a_larger_batch(t):
    """Some rows of quantised activations, with their scales: rows 3 on start at
    no multiple of 16 bytes of scales."""
    wq, sw = codes((1033, 64), 1)[1:], scales(1033, 2)[1:]
    q, s = sa.act_quantize_int8(rows_of((t + 3, 64), torch.bfloat16, 3))
    whole = sa.int8_linear(q, wq, sw, sx=s, dtype=torch.bfloat16)
    assert torch.equal(sa.int8_linear(q[3:], wq, sw, sx=s[3:], dtype=torch.bfloat16), whole[3:])


def test_offsets_past_32_bits():
    """Rows 2^21 entries apart: the last of 1104 lie past 2^31."""
    n, d, ld = 1104, 64, 1 << 21
    far = lambda v: torch.empty(n, ld, dtype=v.dtype, device=DEV)[:, :v.shape[1]].copy_(v)  # noqa: E731
    x = rows_of((n, d), torch.bfloat16, 5)
    q, s = sa.act_quantize_int8(x)
    fq, fs = sa.act_quantize_int8(far(x), xq=far(torch.zeros_like(q)))
    assert torch.equal(fq, q) and torch.equal(fs, s)
    cq, cs = sa.weight_quantize_int8(x[:, :48].contiguous()[:1088])
    fq, fs = sa.weight_quantize_int8(far(x)[:1088, :48])
    assert torch.equal(fq, cq) and torch.equal(fs, cs)
    del fq
    wq, sw = codes((n, d), 6), scales(n, 7)
    fw, fx = far(wq), far(q)
    for t in (1, 4, 8, 40, n):  # a kernel each, and the tiles with rows far apart
        want = sa.int8_linear(q[-t:], wq, sw, sx=s[-t:], dtype=torch.bfloat16)
        assert torch.equal(sa.int8_linear(fx[-t:], fw, sw, sx=s[-t:], dtype=torch.bfloat16), want)


def test_vectors_and_empty():
    wq, sw = codes((40, 64), 1), scales(40, 2)
    x = rows_of((64,), torch.bfloat16, 3)
    y = sa.int8_linear(x, wq, sw)
    q, s = sa.act_quantize_int8(x)
    assert y.shape == (40,) and q.shape == (64,) and s.shape == (1,)
    assert torch.equal(y, sa.int8_linear(x[None], wq, sw)[0])
    assert torch.equal(y, sa.int8_linear(q, wq, sw, sx=s, dtype=torch.bfloat16))
    assert sa.int8_linear(x[None][:0], wq, sw).shape == (0, 40)
    assert sa.int8_linear(q[None][:0], wq, sw, sx=s[:0]).shape == (0, 40)
    q, s = sa.act_quantize_int8(x[None][:0])
    assert q.shape == (0, 64) and s.shape == (0,)


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("t", [1, 6, 70])
def test_a_feed_forward_block(t, dtype):
    """Quantised weights, up and down, beside the dense layer they stand for.
    A code is off by half a step s / 2 = max / 254: an entry of the product by
    sum_k |x| sw / 2 + |w| sx / 2 at most (and their product)."""
    d, f = 264 + 8, 520 + 8
    x, wu, wd = rows_of((t, d), dtype, 1), rows_of((d, f), dtype, 2, 0.06), rows_of((f, d), dtype, 3, 0.06)
    (uq, us), (dq, ds) = sa.weight_quantize_int8(wu), sa.weight_quantize_int8(wd)
    h = sa.int8_linear(x, uq, us, act="silu")
    y = sa.int8_linear(h, dq, ds, residual=x)
    for got, a, w, sw, act, res in ((h, x, wu, us, "silu", None), (y, h, wd, ds, "none", x)):
        A, W, S = f64(a), f64(w), sw.double().cpu().numpy()
        sx = np.abs(A).max(axis=1) / 127 * (1 + E)
        z = A @ W
        off = (np.abs(A).sum(1)[:, None] * S / 2 + np.abs(W).sum(0) * sx[:, None] / 2 + A.shape[1] * sx[:, None] * S / 4) * (1 + 8 * E)
        want = ol.act(act, z) + (0 if res is None else f64(res))
        close(got, want, act_err(z, off + 4 * E * np.abs(z), act) + 4 * E * np.abs(want))


def test_graphs_and_streams():
    dt = torch.bfloat16
    wq, sw = codes((1032, 2064), 1), scales(1032, 2)
    xs = [rows_of((t, 2064), dt, t) for t in (1, 4, 40, 300)]
    want = [sa.int8_linear(x, wq, sw, act="silu") for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(device=DEV) for _ in range(3)]
    got = []
    for _ in range(4):
        for s in streams:
            with torch.cuda.stream(s):
                got.append([sa.int8_linear(x, wq, sw, act="silu") for x in xs])
    torch.cuda.synchronize()
    for g in got:
        assert all(torch.equal(a, b) for a, b in zip(g, want))
    side = streams[0]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        outs = [sa.int8_linear(x, wq, sw, act="silu") for x in xs]
        pairs = [sa.act_quantize_int8(x) for x in xs]
    for k in range(3):
        for i, x in enumerate(xs):
            x.copy_(rows_of(x.shape, dt, 100 * k + i))
        graph.replay()
        torch.cuda.synchronize()
        for x, o, (q, s) in zip(xs, outs, pairs):
            assert torch.equal(o, sa.int8_linear(x, wq, sw, act="silu"))
            same_codes(x, q, s)


def test_python_refusals():
    wq, sw = codes((40, 64), 1), scales(40, 2)
    x, q, s = rows_of((3, 64), torch.float16, 3), codes((3, 64), 4), scales(3, 5)
    for call in (lambda: sa.int8_linear(x.float(), wq, sw), lambda: sa.int8_linear(x, wq.short(), sw),
                 lambda: sa.int8_linear(x, wq.T, sw), lambda: sa.int8_linear(x, wq, sw.double()),
                 lambda: sa.int8_linear(x, wq, sw[:39]), lambda: sa.int8_linear(x, wq, sw, sx=s),
                 lambda: sa.int8_linear(q, wq, sw), lambda: sa.int8_linear(q, wq, sw, sx=s[:2]),
                 lambda: sa.int8_linear(q, wq, sw, sx=s, dtype=torch.float32),
                 lambda: sa.int8_linear(x, wq, sw, dtype=torch.bfloat16), lambda: sa.int8_linear(x.cpu(), wq, sw),
                 lambda: sa.int8_linear(x, wq, sw, bias=sw), lambda: sa.int8_linear(x, wq, sw, act="tanh"),
                 lambda: sa.int8_linear(x, wq, sw, y=torch.empty(3, 40, device=DEV)),
                 lambda: sa.act_quantize_int8(x.float()), lambda: sa.act_quantize_int8(x, xq=q.short()),
                 lambda: sa.act_quantize_int8(x, sx=s[:2]), lambda: sa.weight_quantize_int8(x.T, wq=q)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: sa.act_quantize_int8(x[:, :40].contiguous()), lambda: sa.int8_linear(q[:, 8:56], codes((40, 48), 1), sw, sx=s)):
        with pytest.raises(sa.SparseActError):  # 40 is no multiple of 16; codes not 16-byte aligned
            call()
    x.requires_grad_()
    with pytest.warns(UserWarning, match="no gradient"):
        sa.int8_linear(x, wq, sw)
