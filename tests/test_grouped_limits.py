"""Linear layers grouped by expert at the ends of their sizes, and under choices
of tiles that ordinary calls do not make."""

import pytest
import torch

import sparse_input_gemv_amd as sa
from test_grouped import by_expert, offsets_of
from test_linear import DEV, ints, same

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("with_dbias", [False, True])
def test_the_most_columns_of_the_most_experts(with_dbias):
    """fp16's scales of 512 experts with 2^21 columns: 2^24 blocks of 64 columns."""
    dt, d_in, d_out, counts = torch.float16, 8, 1 << 21, [0] * 512
    for e in (0, 1, 255, 256, 511):
        counts[e] = 2
    T, off = sum(counts), offsets_of(counts)
    x, dy, pre = ints((T, d_in), -2, 2, dt, 1), ints((T, d_out), -1, 1, dt, 2), ints((T, d_out), -3, 3, dt, 3)
    dy[:, 5] *= 2.0**-20  # a column that is scaled
    wt = torch.empty(1, d_in, d_out, dtype=dt, device=DEV).expand(512, d_in, d_out)
    _, dwt, db = sa.grouped_linear_backward(dy, x, wt, off, act="relu", pre=pre, with_dx=False, with_dbias=with_dbias)
    at = torch.ones(512, dtype=torch.bool, device=DEV)
    for e, r in by_expert(counts):
        d = dy[r].double() * (pre[r] > 0).double()
        same(dwt[e], x[r].double().T @ d)
        if with_dbias:
            same(db[e], d.sum(0))
        at[e] = False
    for e in at.nonzero()[:, 0].tolist():
        assert not dwt[e].any() and (db is None or not db[e].any())
