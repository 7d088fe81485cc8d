"""Linear layers grouped by expert at the ends of their sizes, and under choices
of tiles that ordinary calls do not make."""

import pytest
import torch

import sparse_input_gemv_amd as sa
from test_grouped import by_expert, offsets_of
from test_linear import DEV, ints, same
from test_linear import tuning  # noqa: F401

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


def kernels_of(call):
    """Names of the kernels that a call launches."""
    with torch.profiler.profile(activities=[torch.profiler.ProfilerActivity.CUDA]) as p:
        call()
        torch.cuda.synchronize()
    return [e.name for e in p.events() if "k_grp<" in e.name]


def test_weight_gradients_follow_their_own_tiles(tuning):  # noqa: F811
    """Choices that weight gradients do not have (64 rows and fewer, 256 x 192)
    leave their tile automatic: 256 x 256 for many rows of few experts, else 128
    x 128."""
    dt, wanted = torch.bfloat16, {-1: (256, 128), 0: (256, 256), 1: (128, 128), 2: (256, 128), 5: (256, 128)}
    for k, (t, d) in enumerate(((4096, 4096), (64, 256))):
        x, dy, wt = ints((t, d), -2, 2, dt, 1), ints((t, d), -1, 1, dt, 2), ints((1, d, d), -2, 2, dt, 3)
        off, want = offsets_of([t]), x.double().T @ dy.double()
        for tile, rows in wanted.items():
            tuning(tile)
            out = []
            names = kernels_of(lambda: out.append(sa.grouped_linear_backward(dy, x, wt, off, with_dx=False)[1]))
            assert len(names) == 1 and f"{rows[k]}, {rows[k]}, 2, 2, 2>" in names[0], (tile, names)
            same(out[0][0], want)
