"""What the block operators do under torch's autograd beyond first derivatives."""
import pytest
import torch

from test_gpu_blocks import gen, norm_inputs, nss, randn, rotary_inputs      # noqa: F401  (nss is a fixture)

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- second derivatives

@pytest.mark.parametrize("linear", [False, True])
@pytest.mark.parametrize("wrt", ["x", "weight", "bias"])
def test_layer_norm_refuses_a_second_derivative(nss, linear, wrt):
    """Also where the gradient that arrives is a constant (a linear loss), so that only x and weight carry a graph."""
    from newton_schulz_stacked_gb300 import autograd as A
    x, w, b, t = norm_inputs(1, 12, 48, torch.float32, torch.float32)
    leaf = {"x": x.requires_grad_(), "weight": w.requires_grad_(), "bias": b.requires_grad_()}
    y = A.layer_norm(x, w, b)
    loss = (y * t).sum() if linear else y.square().sum()
    g, = torch.autograd.grad(loss, leaf[wrt], create_graph=True)
    if wrt == "bias" and linear:
        want = t.sum(0)                                       # the first derivative stays usable
        assert torch.allclose(g, want, rtol=0, atol=1e-5)
    with pytest.raises(RuntimeError, match="second derivative"):
        (loss + g.square().sum()).backward()


@pytest.mark.parametrize("linear", [False, True])
@pytest.mark.parametrize("normalize", [False, True])
def test_route_refuses_a_second_derivative(nss, linear, normalize):
    from newton_schulz_stacked_gb300 import autograd as A
    g = gen(2)
    logits = randn(g, 30, 12).requires_grad_()
    r = A.route(logits, 3, normalize=normalize)
    for loss in (r.loss if linear else r.loss.square(), (r.gate * 2).sum() if linear else r.gate.square().sum()):
        d, = torch.autograd.grad(loss, logits, create_graph=True)
        with pytest.raises(RuntimeError, match="second derivative"):
            (loss + d.square().sum()).backward(retain_graph=True)


def test_first_derivatives_with_a_graph_are_the_same(nss):
    from newton_schulz_stacked_gb300 import autograd as A
    x, w, b, t = norm_inputs(3, 12, 48, torch.float32, torch.float32)
    leaves = [v.requires_grad_() for v in (x, w, b)]
    loss = (A.layer_norm(*leaves) * t).sum()
    for a, c in zip(torch.autograd.grad(loss, leaves, create_graph=True), torch.autograd.grad(loss, leaves)):
        assert torch.equal(a, c)


@pytest.mark.parametrize("with_k", [True, False])
def test_rotary_second_derivative(nss, with_k):
    """The rotation is linear, so its gradient is a rotation that has a gradient: a penalty on it against 64 bits."""
    from newton_schulz_stacked_gb300 import autograd as A
    q, k, pos, freq = rotary_inputs(4, 2, 7, 3, 1, 20, (4, 6), torch.float32)
    axis = torch.repeat_interleave(torch.arange(2), torch.tensor((4, 6))).cuda()
    angle = (pos.float()[axis].permute(1, 2, 0) * freq).double()[:, :, None]

    def turned(z):
        u, v = z[..., :10], z[..., 10:]
        return torch.cat((u * angle.cos() - v * angle.sin(), v * angle.cos() + u * angle.sin()), -1)

    def penalised(rot, leaves):
        outs = rot(leaves)
        loss = sum((o ** 3).sum() for o in outs)
        grads = torch.autograd.grad(loss, leaves, create_graph=True)
        (loss + sum(((g * 0.5) ** 2).sum() for g in grads)).backward()
        return [p.grad for p in leaves]

    point = (q, k) if with_k else (q,)
    got = penalised(lambda z: [o for o in A.rotary(z[0], z[1] if with_k else None, pos, freq, (4, 6)) if o is not None],
                    [z.clone().requires_grad_() for z in point])
    want = penalised(lambda z: [turned(o) for o in z], [z.double().requires_grad_() for z in point])
    for a, c in zip(got, want):
        # three rotations of 8 U each, products of up to three rounded factors
        assert ((a.double() - c).abs() <= 100 * 2.0 ** -24 * (c.abs() + c.abs().amax())).all()


def test_negated_gradients(nss):
    """A gradient that comes through a conjugate's imaginary part may be a negated view."""
    from newton_schulz_stacked_gb300 import autograd as A

    def minus(t):
        return torch.complex(torch.zeros_like(t), t).conj().imag

    def grads(f, *leaves):
        return torch.autograd.grad(f(*leaves), leaves)

    q, k, pos, freq = rotary_inputs(5, 1, 3, 2, 1, 8, (4,), torch.float32)
    logits = randn(gen(6), 9, 4).requires_grad_()
    x, w, b, _ = norm_inputs(7, 1, 1, torch.float32, torch.float32)
    leaves = [v.requires_grad_() for v in (x, w, b)]
    for f, at in ((lambda l: A.route(l, 2).loss, [logits]), (lambda l: A.route(l[:1], 1).gate, [logits]),
                  (lambda *v: A.layer_norm(*v), leaves),
                  (lambda a: A.rotary(a, None, pos, freq, (4,))[0], [q.requires_grad_()])):
        for a, c in zip(grads(lambda *v: minus(f(*v)).sum(), *at), grads(lambda *v: -f(*v).sum(), *at)):
            assert torch.equal(a, c)
