"""Plans of split products at sizes whose reduction no launch could hold (on the
CPU: plans compute nothing)."""

import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "sparse_input_gemv_amd", "libsparse_act.so")


@pytest.mark.skipif(not os.path.exists(LIB), reason="library not built")
def test_splits_have_fewer_outputs_than_a_launch_has_threads():
    import sparse_input_gemv_amd as m

    m.set_linear_tuning(0, 8)
    try:
        assert m.linear_plan("forward", 1 << 18, 64, 1 << 14)["split"] == 8
        # 2^34 outputs, four to a thread: 2^32 threads
        for op in ("forward", "gated"):
            assert m.linear_plan(op, 1 << 20, 64, 1 << 14)["split"] == 0
        assert m.linear_plan("dx", 1 << 20, 1 << 14, 64)["split"] == 0
        assert m.linear_plan("gated_dw", 64, 1 << 17, 1 << 16)["split"] == 0
        assert m.lib().int8_linear_workspace_bytes(1 << 18, 64, 1 << 14, 1) > 0
        assert m.lib().int8_linear_workspace_bytes(1 << 20, 64, 1 << 14, 1) == 0
    finally:
        m.set_linear_tuning()
