"""The one-launch sum of the dense linear layers' split products: which streams
keep counters for it, and calls that use them at every tile height."""

import ctypes

import numpy as np
import pytest
import torch

import sparse_input_gemv_amd as sa
from test_linear import DEV, ints, layer_inputs, same

# torch's stream ids as (id, handle, whether the id names one stream for good)
IDS = [(0, 0, True), (3, 94697688000608, True), (995, 94697699987664, True),  # default, pooled
       (94697688738592, 94697688738592, False),                               # an external stream
       (2, 2, False), (1, 1, False),                                          # per-thread, legacy handles
       (0, 94697688738592, False)]


@pytest.mark.parametrize("sid, handle, lasting", IDS)
def test_streams_that_keep_counters(sid, handle, lasting):
    assert sa._lasting(sid, handle) is lasting


def split_call(i):
    return (sa.dense_linear(i[0], i[1], act="silu"), *sa.gated_linear(i[0], i[1], i[2], with_gu=True))


@pytest.mark.gpu
@pytest.mark.parametrize("t", [1, 16])
def test_external_streams_keep_no_counters(t):
    """A stream that torch did not make, destroyed and made again: equal bits,
    and nothing is kept under its handle."""
    ins = layer_inputs(t, 2056, 1032, 21, torch.float16)
    assert sa.linear_plan("forward", t, 2056, 1032)["split"] > 0
    want = split_call(ins)
    torch.cuda.synchronize()
    kept = dict(sa._tickets)
    rt = torch.cuda.cudart()
    for _ in range(3):
        h = ctypes.c_void_p()
        assert int(rt.cudaStreamCreate(ctypes.addressof(h))) == 0
        stream = torch.cuda.ExternalStream(h.value, device=DEV)
        with torch.cuda.stream(stream):
            for _ in range(3):
                got = split_call(ins)
        stream.synchronize()
        assert int(rt.cudaStreamDestroy(h.value)) == 0
        for a, b in zip(got, want):
            assert torch.equal(a, b)
        assert sa._tickets.keys() == kept.keys()


def one_launch(op, t, d_in, d_out):
    """Whether a call with counters sums its shares in the same launch."""
    p = sa.linear_plan(op, t, d_in, d_out)
    rounds = -(-min(t, p["tile_rows"]) // 16) * (p["split"] // p["tiles"] // 4 + 1)
    return p["split"] > 0 and p["tile_rows"] <= 64 and p["tiles"] <= 512 and rounds <= 4


def test_the_documented_examples():
    for op in ("forward", "gated"):
        for t in (1, 16):
            assert one_launch(op, t, 4096, 4096)
        for t in (17, 64):
            assert one_launch(op, t, 4096, 14336)
        assert not one_launch(op, 33, 4096, 1024) and not one_launch(op, 64, 4096, 4096)


D_IN, D_OUT = 1032, 8456  # a ragged last step and last tile


@pytest.mark.gpu
@pytest.mark.parametrize("t, tile_rows", [(1, 16), (16, 16), (17, 32), (30, 32), (33, 64), (64, 64)])
def test_one_launch_on_streams_at_once_and_beside_graphs(t, tile_rows):
    """Eager calls that add their partial sums within the launch, on three
    streams at once, beside a replayed graph of the same calls (which take the
    second launch): the fp64 result rounded once, and equal bits."""
    for op in ("forward", "gated"):
        assert one_launch(op, t, D_IN, D_OUT)
        assert sa.linear_plan(op, t, D_IN, D_OUT)["tile_rows"] == tile_rows
    dt = torch.bfloat16
    wg, wu = ints((D_IN, D_OUT), -2, 2, dt, 31), ints((D_IN, D_OUT), -1, 1, dt, 32)
    xs = [ints((t, D_IN), -2, 2, dt, 40 + k) for k in range(3)]
    f = lambda x: (sa.dense_linear(x, wg), *sa.gated_linear(x, wg, wu, act="relu", with_gu=True))  # noqa: E731
    want = []
    for x in xs:
        g64, u64 = x.double() @ wg.double(), x.double() @ wu.double()
        got = f(x)
        for a, b in zip(got, (g64, g64.clamp(min=0) * u64, g64, u64)):
            same(a, b)
        want.append(got)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = f(xs[1])
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    for _ in range(6):
        for v in out:
            v.zero_()
        torch.cuda.synchronize()
        got = []
        for k in range(4):
            for x, s in zip(xs, streams):
                with torch.cuda.stream(s):
                    got.append(f(x))
            if k == 1:
                graph.replay()
        torch.cuda.synchronize()
        for k, g in enumerate(got + [out]):
            for a, b in zip(g, want[1 if g is out else k % 3]):
                assert torch.equal(a, b)
    for s in streams:  # the counters are left zero
        tk = sa._tickets.get((0, s.stream_id))
        assert tk is not None and not tk.any()


@pytest.mark.gpu
@pytest.mark.parametrize("t", [17, 33, 64])
def test_one_launch_of_real_values(t):
    """Real values: the bits of the one launch are the captured call's."""
    gen = np.random.default_rng(t)
    to = lambda a: torch.from_numpy(a).to(torch.float16).to(DEV)  # noqa: E731
    x, w = to(gen.standard_normal((t, D_IN))), to(0.05 * gen.standard_normal((D_IN, D_OUT)))
    b = to(gen.standard_normal(D_OUT))
    f = lambda: (sa.dense_linear(x, w, bias=b, act="gelu"), *sa.gated_linear(x, w, w, with_gu=True))  # noqa: E731
    f()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = f()
    for _ in range(4):
        for v in out:
            v.zero_()
        graph.replay()
        for a, c in zip(f(), out):
            assert torch.equal(a, c)
