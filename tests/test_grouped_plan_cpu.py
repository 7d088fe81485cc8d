"""Plans of the products grouped by expert, as the C header states them (plans
compute nothing on the GPU)."""

import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "sparse_input_gemv_amd", "libsparse_act.so")
pytestmark = pytest.mark.skipif(not os.path.exists(LIB), reason="library not built")

OPS = ("forward", "gated", "dx", "gated_dx")
SHAPES = [(1, 8, 4096, 4096), (16, 8, 4096, 14336), (509, 16, 1024, 4096), (1000, 64, 1024, 4096), (4096, 8, 4096, 11008),
          (8192, 8, 14336, 4096)]


@pytest.fixture
def sa():
    import sparse_input_gemv_amd as m
    yield m
    m.set_linear_tuning()


def plans(sa):
    return [sa.grouped_plan(op, *s) for op in OPS for s in SHAPES]


@pytest.mark.parametrize("split", [-1, 0, 8, 512])
def test_tile_5_counts_as_automatic(sa, split):
    sa.set_linear_tuning(-1, split)
    want = plans(sa)
    sa.set_linear_tuning(5, split)
    assert plans(sa) == want


def test_tiles_of_256_rows_are_split_from_24_steps_on(sa):
    sa.set_linear_tuning(0)
    for op, d_in, d_out, per in (("forward", 64, 4096, 1), ("gated", 64, 4096, 1), ("dx", 4096, 64, 1), ("gated_dx", 4096, 64, 2)):
        for steps in (22, 23, 24, 26):
            if steps % per:
                continue
            k = steps // per
            plan = sa.grouped_plan(op, 8192, 8, d_in * (k if d_in == 64 else 1), d_out * (k if d_out == 64 else 1))
            assert plan == {"tile_rows": 256, "split": 256 if steps >= 24 else 0}
    sa.set_linear_tuning(0, 0)
    assert sa.grouped_plan("forward", 8192, 8, 4096, 4096)["split"] == 0
    sa.set_linear_tuning(0, 8)  # set by hand: whatever the steps
    assert sa.grouped_plan("forward", 8192, 8, 64, 4096) == {"tile_rows": 256, "split": 8}
    sa.set_linear_tuning(0, 512)  # one share per compute unit at most
    assert sa.grouped_plan("forward", 8192, 8, 4096, 4096) == {"tile_rows": 256, "split": 256}


def test_scratch_of_shares(sa):
    """Two tiles of fp32 per share and 32 bytes: 128 MiB for 256 shares of 256 x
    256, whatever the rows."""
    need = [sa.lib().grouped_linear_workspace_bytes(T, 8, 4096, 4096) for T in (4096, 8192, 1 << 20)]
    assert need == [256 * 32 + 256 * 2 * 256 * 256 * 4] * 3
    sa.set_linear_tuning(-1, 0)
    assert sa.lib().grouped_linear_workspace_bytes(8192, 8, 4096, 4096) == 0
