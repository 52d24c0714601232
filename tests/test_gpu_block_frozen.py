"""Layer norm gradients with some of the parameters' gradients left out."""
import pytest
import torch

from test_gpu_blocks import TYPES, check_norm_backward, norm_inputs, nss, same_bits      # noqa: F401  (nss is a fixture)

pytestmark = pytest.mark.gpu

# every kernel of the backward pass
SHAPES = [(3, 40), (400, 96), (700, 201), (500, 768), (400, 777), (300, 2048), (300, 2051), (90, 8192), (90, 8200), (90, 8203)]


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("dtype,wtype", [("bf16", "f32"), ("f16", "f16"), ("f32", "f32")])
def test_gradients_that_are_not_wanted(nss, rows, cols, dtype, wtype):
    x, w, b, dy = norm_inputs(rows + cols, rows, cols, TYPES[dtype], TYPES[wtype])
    _, mean, rstd = nss.mb_layer_norm(x, w, b)
    dx, dw, db = check_norm_backward(nss, dy, x, mean, rstd, w)
    for weight_grad in (True, False):
        for bias in (True, False):
            before = nss.mb_launch_count()
            got = nss.mb_layer_norm_backward(dy, x, mean, rstd, w, bias=bias, weight_grad=weight_grad)
            launches = nss.mb_launch_count() - before
            same_bits(got[0], dx, "dx")
            for g, want, wanted in ((got[1], dw, weight_grad), (got[2], db, bias)):
                assert (g is not None) == wanted
                if wanted:
                    same_bits(g, want, f"of {weight_grad, bias}")
            assert launches == 1 if not (bias or weight_grad) else launches >= 1
    # a given result is wanted, whatever the flags say
    given = torch.empty_like(dw), torch.empty_like(db)
    nss.mb_layer_norm_backward(dy, x, mean, rstd, w, bias=False, weight_grad=False, dweight=given[0], dbias=given[1])
    same_bits(given[0], dw, "given dweight")
    same_bits(given[1], db, "given dbias")


@pytest.mark.parametrize("rows,cols", SHAPES)
def test_a_bias_without_a_weight(nss, rows, cols):
    """The forward call takes a bias alone; its gradient goes to a result that the caller passes, in x's type or fp32."""
    x, _, b, dy = norm_inputs(rows + cols, rows, cols, torch.bfloat16, torch.float32)
    _, mean, rstd = nss.mb_layer_norm(x, None, b)
    plain = check_norm_backward(nss, dy, x, mean, rstd, None)
    assert plain[1] is None and plain[2] is None
    for dtype in (torch.float32, torch.bfloat16):
        want = nss.mb_layer_norm_backward(dy, x, mean, rstd, torch.ones(cols, device="cuda", dtype=dtype))
        db = torch.empty(cols, device="cuda", dtype=dtype)
        got = nss.mb_layer_norm_backward(dy, x, mean, rstd, None, dbias=db)
        assert got[1] is None and got[2] is db
        same_bits(db, want[2], "dbias")
        same_bits(got[0], plain[0], "dx")
    for wrong in (torch.empty(cols, device="cuda", dtype=torch.float16), torch.empty(cols + 1, device="cuda")):
        with pytest.raises(ValueError):
            nss.mb_layer_norm_backward(dy, x, mean, rstd, None, dbias=wrong)
    with pytest.raises(ValueError):
        nss.mb_layer_norm_backward(dy, x, mean, rstd, None, dweight=torch.empty(cols, device="cuda"))


@pytest.mark.parametrize("train_w", [True, False])
@pytest.mark.parametrize("train_b", [True, False])
def test_frozen_parameters_under_autograd(nss, train_w, train_b):
    from newton_schulz_stacked_gb300 import autograd as A
    x, w, b, t = norm_inputs(3, 400, 768, torch.bfloat16, torch.float32)
    x.requires_grad_()
    w.requires_grad_(train_w), b.requires_grad_(train_b)
    y = A.layer_norm(x, w, b)
    _, mean, rstd = nss.mb_layer_norm(x.detach(), w.detach(), b.detach())
    want = nss.mb_layer_norm_backward(t, x.detach(), mean, rstd, w.detach())
    before = nss.mb_launch_count()
    got = torch.autograd.grad(y, [v for v in (x, w, b) if v.requires_grad], t)
    launches = nss.mb_launch_count() - before
    for a, c in zip(got, [g for g, v in zip(want, (x, w, b)) if v.requires_grad]):
        same_bits(a, c, "gradient")
    # autograd may run a backward pass in a thread of its own, whose launches are counted there
    assert launches in ((0, 2) if train_w or train_b else (0, 1))
