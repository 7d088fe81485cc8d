"""The dense linear layers stand outside autograd, and say so: a forward call
with inputs that require grad warns, and its values are those of any call."""

import warnings

import pytest
import torch

import sparse_input_gemv_amd as sa


def silent(f, *args):
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        return f(*args)


def test_the_warning():
    a, b = torch.zeros(2), torch.zeros(2, requires_grad=True)
    silent(sa._lin_detached, "dense_linear", a, a, None)
    with pytest.warns(UserWarning, match="dense_linear is outside autograd.*dense_linear_backward"):
        sa._lin_detached("dense_linear", a, None, b)
    with torch.no_grad():
        silent(sa._lin_detached, "dense_linear", b)
    with torch.inference_mode():
        silent(sa._lin_detached, "gated_linear", b)


@pytest.mark.gpu
@pytest.mark.parametrize("t", [1, 40])
def test_forward_calls_warn_where_gradients_would_be_lost(t):
    gen = torch.Generator(device="cuda").manual_seed(3)
    mk = lambda *s: torch.randn(*s, generator=gen, device="cuda").to(torch.bfloat16)  # noqa: E731
    x, w, b, r = mk(t, 136), mk(136, 264), mk(264), mk(t, 264)
    y, h = silent(sa.dense_linear, x, w, b, "silu", r), silent(sa.gated_linear, x, w, w)
    for k in range(4):
        ins = [v.clone().requires_grad_(i == k) for i, v in enumerate((x, w, b, r))]
        with pytest.warns(UserWarning, match="outside autograd"):
            got = sa.dense_linear(ins[0], ins[1], ins[2], "silu", ins[3])
        assert torch.equal(got, y) and not got.requires_grad
        with torch.no_grad():
            assert torch.equal(silent(sa.dense_linear, ins[0], ins[1], ins[2], "silu", ins[3]), y)
    p = torch.nn.Parameter(w)
    with pytest.warns(UserWarning, match="gated_linear_backward"):
        assert torch.equal(sa.gated_linear(x, p, w), h)
    # the backward calls are the gradients: parameters are their ordinary arguments
    dx, dw, db = silent(sa.dense_linear_backward, r, x, p, "none", None, True)
    want = sa.dense_linear_backward(r, x, w, with_dbias=True)
    assert all(torch.equal(a, c) and not a.requires_grad for a, c in zip((dx, dw, db), want))
