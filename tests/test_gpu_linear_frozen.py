"""autograd.linear with some of its inputs frozen: what no wanted gradient reads is not kept, and second derivatives still raise."""
import itertools

import pytest
import torch

from test_gpu_linear import _gen, _rows, nss      # noqa: F401  (nss is a fixture)

pytestmark = pytest.mark.gpu

ROWS, COLS, OUT = 90, 72, 136


def _leaves(groups, act, seed=0):
    g, t = _gen(61 + seed), torch.bfloat16
    shape = (groups, OUT, COLS) if groups else (OUT, COLS)
    x = _rows(ROWS, COLS, t, g)
    w = (torch.randn(shape, generator=g, device="cuda") * COLS ** -0.5).to(t)
    b, r, dy = torch.randn(shape[:-1], generator=g, device="cuda"), _rows(ROWS, OUT, t, g), _rows(ROWS, OUT, t, g)
    ends = torch.tensor([30, 30, 80], dtype=torch.int32, device="cuda") if groups else None
    return x, w, b, r, dy, ends


@pytest.mark.parametrize("groups", [0, 3])
@pytest.mark.parametrize("act", ["none", "gelu"])
def test_any_gradients_that_are_wanted(nss, groups, act):
    """Every choice of x, weight, bias and residual: the bits of the call that wants all."""
    from newton_schulz_stacked_gb300 import autograd
    x, w, b, r, dy, ends = _leaves(groups, act)
    full = [t.clone().requires_grad_() for t in (x, w, b, r)]
    autograd.linear(*full, act, ends).backward(dy)
    for want in itertools.product((False, True), repeat=4):
        if not any(want):
            continue
        leaves = [t.clone().requires_grad_(g) for t, g in zip((x, w, b, r), want)]
        y = autograd.linear(*leaves, act, ends)
        # inputs that no wanted gradient reads may change before the backward pass
        with torch.no_grad():
            if not want[1]:
                leaves[0].fill_(float("nan"))
            if not want[0]:
                leaves[1].fill_(float("nan"))
            leaves[2].fill_(float("nan"))
        y.backward(dy)
        for i, (leaf, ref, wanted) in enumerate(zip(leaves, full, want)):
            assert (leaf.grad is not None) == wanted
            if wanted:                           # (a product alone may be cut otherwise than both)
                torch.testing.assert_close(leaf.grad, ref.grad, rtol=2.0 ** -7, atol=2.0 ** -7)


def test_what_is_not_read_is_not_kept(nss):
    from newton_schulz_stacked_gb300 import autograd
    x, w, b, r, dy, _ = _leaves(0, "gelu")
    for train_w in (False, True):
        inner = x.clone().requires_grad_() * 1.0                  # x of an earlier operation
        y = autograd.linear(inner, w.clone().requires_grad_(train_w), None, None, "gelu")
        kept = [t for t in y.grad_fn.saved_tensors if t is not None and t.data_ptr() == inner.data_ptr()]
        assert len(kept) == train_w
    # what is read is still guarded
    leaf = x.clone().requires_grad_()
    weight = w.clone()
    y = autograd.linear(leaf, weight, None, None, "gelu")
    weight.zero_()
    with pytest.raises(RuntimeError, match="modified"):
        y.backward(dy)


@pytest.mark.parametrize("frozen", ["x", "weight", "none"])
def test_second_derivatives_raise(nss, frozen):
    """Through z, whichever inputs are kept: none is taken for a constant."""
    from newton_schulz_stacked_gb300 import autograd
    x, w, b, _, dy, _ = _leaves(0, "gelu")
    x.requires_grad_(frozen != "x")
    w.requires_grad_(frozen != "weight")
    b.requires_grad_()
    y = autograd.linear(x, w, b, None, "gelu")
    leaves = [t for t in (x, w, b) if t.requires_grad]
    grads = torch.autograd.grad(y, leaves, dy, create_graph=True)
    for g, leaf in itertools.product(grads, leaves):
        with pytest.raises(RuntimeError, match="second"):
            torch.autograd.grad(g.float().sum(), leaf, retain_graph=True)


def test_backward_calls_without_what_they_do_not_read(nss):
    for groups in (0, 3):
        x, w, b, _, dy, ends = _leaves(groups, "silu")
        _, z = nss.mb_linear(x, w, b, None, "silu", ends, keep=True)
        dx, _, _ = nss.mb_linear_backward(dy, x, w, z, "silu", ends, weight_grad=False)
        _, dw, db = nss.mb_linear_backward(dy, x, w, z, "silu", ends, input_grad=False, bias=True)
        got, none, _ = nss.mb_linear_backward(dy.view(9, 10, OUT), None, w, z.view(9, 10, OUT), "silu", ends, weight_grad=False)
        assert got.shape == (9, 10, COLS) and none is None and torch.equal(got.view(ROWS, COLS), dx)
        _, got, got_b = nss.mb_linear_backward(dy, x, None, z, "silu", ends, input_grad=False, bias=True)
        assert torch.equal(got, dw) and torch.equal(got_b, db)
        _, _, got = nss.mb_linear_backward(dy, None, None, z, "silu", ends, input_grad=False, weight_grad=False, bias=True)
        torch.testing.assert_close(got, db, rtol=2.0 ** -7, atol=2.0 ** -7)
        for wrong, match in (((None, w), "needs x"), ((x, None), "needs the weight")):
            with pytest.raises(ValueError, match=match):
                nss.mb_linear_backward(dy, *wrong, z, "silu", ends)
        with pytest.raises(ValueError, match="dy"):
            nss.mb_linear_backward(dy[:, :-1].contiguous(), None, w, z, "silu", ends, weight_grad=False)
        with pytest.raises(ValueError, match="x"):
            nss.mb_linear_backward(dy, x.half(), None, z, "silu", ends, input_grad=False)
        if groups:
            with pytest.raises(ValueError, match="ends"):
                nss.mb_linear_backward(dy, x, None, z, "silu", ends.long(), input_grad=False)


def test_z_is_formed_for_a_backward_pass_only(nss, monkeypatch):
    """Parameters that require gradients, evaluated without recording: no second result is written."""
    from newton_schulz_stacked_gb300 import autograd
    x, w, b, r, _, ends = _leaves(3, "silu")
    w.requires_grad_()
    kept, call = [], autograd._k.mb_linear

    def seen(*args, keep, **more):
        kept.append(keep)
        return call(*args, keep=keep, **more)

    monkeypatch.setattr(autograd._k, "mb_linear", seen)
    want = autograd.linear(x, w, b, r, "silu", ends)
    with torch.no_grad():
        assert torch.equal(autograd.linear(x, w, b, r, "silu", ends), want)
    with torch.inference_mode():
        assert torch.equal(autograd.linear(x, w, b, r, "silu", ends), want)
    autograd.linear(x, w, b, r, "none", ends)
    autograd.linear(x, w.detach(), b, r, "silu", ends)
    assert kept == [True, False, False, False, False]
