"""The one-launch sum of the dense linear layers' split products: which streams
keep counters for it, and calls that use them at every tile height."""

import ctypes

import pytest
import torch

import sparse_input_gemv_amd as sa
from test_linear import DEV, layer_inputs

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
