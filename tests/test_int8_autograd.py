"""The 8-bit layers stand outside autograd and say so, each of them."""

import warnings

import pytest
import torch

import sparse_input_gemv_amd as sa
from test_int8 import codes, rows_of, scales

pytestmark = pytest.mark.gpu


def calls():
    x, wt = rows_of((3, 64), torch.bfloat16, 1), rows_of((64, 40), torch.bfloat16, 2)
    q, wq, sx, sw = codes((3, 64), 3), codes((40, 64), 4), scales(3, 5), scales(40, 6)
    b, r = rows_of((40,), torch.bfloat16, 7), rows_of((3, 40), torch.bfloat16, 8)
    product = lambda i, t: sa.int8_linear(q, wq, t[1], sx=t[0], bias=t[2], residual=t[3], dtype=torch.bfloat16)  # noqa: E731
    return [("act_quantize_int8", lambda i, t: sa.act_quantize_int8(t[0]), [x], 0),
            ("weight_quantize_int8", lambda i, t: sa.weight_quantize_int8(t[0]), [wt], 0),
            ("int8_linear", lambda i, t: sa.int8_linear(t[0], wq, sw), [x], 0)] \
        + [("int8_linear", product, [sx, sw, b, r], i) for i in range(4)]


@pytest.mark.parametrize("k", range(7))
def test_inputs_that_require_grad_bring_a_warning(k):
    name, call, inputs, i = calls()[k]
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        call(i, inputs)
    inputs[i].requires_grad_()
    with pytest.warns(UserWarning, match=f"{name} is outside autograd and has no gradient") as seen:
        out = call(i, inputs)
    assert seen[0].filename == __file__  # the caller's line
    assert not any(t.requires_grad for t in (out if isinstance(out, tuple) else (out,)))
    with warnings.catch_warnings(), torch.no_grad():
        warnings.simplefilter("error")
        call(i, inputs)
