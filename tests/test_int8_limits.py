"""Linear layers in 8-bit integers at the ends of their ranges: codes, scales
and sizes that the calls accept and ordinary layers do not reach."""

import numpy as np
import pytest
import torch

import sparse_input_gemv_amd as sa
from test_int8 import codes, rows_of, scales
from test_linear import DEV, E, close, f64
from test_linear import tuning  # noqa: F401

pytestmark = pytest.mark.gpu
# tokens, tile, split: 16 channels per workgroup, then every tile whole and shared
KERNELS = [(1, -1, -1), (40, -1, -1), (70, -1, -1)] + [(300, tile, split) for tile in range(6) for split in (0, 64)]


def check(x, sx, wq, sw, bias=None):
    """As test_int8's, the sums taken in fp64 on the GPU (exact below 2^53)."""
    y = sa.int8_linear(x, wq, sw, sx=sx, bias=bias, dtype=torch.bfloat16)
    prod = ((x.double() @ wq.double().T) * sw.double() * sx.double()[:, None]).cpu().numpy()
    want = prod if bias is None else prod + f64(bias)
    # past bf16's range the definition rounds to Inf; below it, to a multiple of
    # 2^-133: half a step is 2^-134, and the fp32 products' underflow 2^-150 each
    over = abs(want) >= 2.0**128 * (1 - 2.0**-9)
    assert (f64(y)[over] == np.sign(want[over]) * np.inf).all()
    close(y[torch.from_numpy(~over).to(DEV)], want[~over], (2 * E * abs(prod) + 4 * E * abs(want) + 2.0**-133)[~over])
    return y


@pytest.mark.parametrize("t, tile, split", KERNELS)
def test_sums_of_two_to_the_31(tuning, t, tile, split):  # noqa: F811
    """Codes of -128 in both operands of the longest sum: 2^17 products of 2^14
    are 2^31, which 32 bits hold as -2^31 alone."""
    tuning(tile, split)
    d_in, d_out = 131072, 136
    x, wq = codes((t, d_in), 1), codes((d_out, d_in), 2)
    x[t // 2], x[0], x[t - 1] = 127, -128, -128
    wq[0], wq[1], wq[2], wq[d_out - 1] = -128, 127, 0, -128
    one = torch.ones(t, device=DEV)
    for bias in (None, rows_of((d_out,), torch.bfloat16, 3)):
        y = check(x, one, wq, torch.full((d_out,), 2.0**-8, device=DEV), bias=bias)
    assert (y[t - 1, [0, d_out - 1]] > 0).all() and (y[t - 1, 1] < 0)


def test_the_most_rows_of_1024_threads():
    """2^22 rows of over 16384 values, 1024 threads each: 2^32 threads, which no
    single launch has.  206 GB; only the rows that are compared are written."""
    T, d = 1 << 22, 16400
    if torch.cuda.mem_get_info()[0] < 3 * T * d + (8 << 30):
        torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 3 * T * d + (8 << 30):
        pytest.skip("needs 215 GB of the GPU's memory")
    x = torch.empty(T, d, dtype=torch.bfloat16, device=DEV)
    parts = [slice(0, 3), slice(T // 2 - 2, T // 2 + 2), slice(T - 3, T)]
    for k, r in enumerate(parts):
        x[r] = rows_of((r.stop - r.start, d), torch.bfloat16, k)
    q, s = sa.act_quantize_int8(x)
    for r in parts:
        wq, ws = sa.act_quantize_int8(x[r])
        assert torch.equal(q[r], wq) and torch.equal(s[r], ws)
    del x, q, s
    torch.cuda.empty_cache()


@pytest.mark.parametrize("t, tile, split", [(2, -1, -1), (6, -1, -1)] + KERNELS[1:])
def test_scales_of_any_size_up_to_two_to_the_96(tuning, t, tile, split):  # noqa: F811
    """The sum times the channel's scale is formed first: a channel of 2^96 and
    one of 2^-126 beside ordinary ones, tokens' scales as far apart."""
    tuning(tile, split)
    d_in, d_out = 4112, 136
    x, wq, sw, sx = codes((t, d_in), 1), codes((d_out, d_in), 2), scales(d_out, 3), scales(t, 4)
    x[0], wq[:3] = 127, 127
    sw[0], sw[1], sw[2] = 2.0**96, 2.0**-126, 2.0**60
    sx[0], sx[t - 1] = 2.0**-110, 2.0**60
    y = check(x, sx, wq, sw)
    assert torch.isfinite(y[0]).all() and (y[0, :1] > 2.0**8).all()
    sx[0], sw[0] = 2.0**96, 2.0**-110
    check(x, sx, wq, sw)
