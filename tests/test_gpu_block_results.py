"""Results that the caller passes, and tensors that are views torch has not carried out."""
import pytest
import torch

from test_gpu_blocks import gen, norm_inputs, nss, randn, rotary_inputs, same_bits      # noqa: F401  (nss is a fixture)

pytestmark = pytest.mark.gpu


def _given(nss):
    """name -> (call with results passed, the results)"""
    x, w, b, dy = norm_inputs(1, 40, 96, torch.bfloat16, torch.float32)
    y, mean, rstd = nss.mb_layer_norm(x, w, b)
    q, k, pos, freq = rotary_inputs(2, 2, 9, 3, 1, 32, (16,), torch.float32)
    logits = randn(gen(3), 50, 16)
    r = nss.mb_router(logits, 2)
    new = torch.empty_like
    norm = dict(y=new(y), mean=new(mean), rstd=new(rstd))
    back = dict(dx=new(x), dweight=new(w), dbias=new(b))
    rot = dict(q_out=new(q), k_out=new(k))
    route = {n: new(v) for n, v in r._asdict().items()}
    dlogits = dict(dlogits=new(logits))
    one = torch.ones(1, device="cuda")
    return {
        "mb_layer_norm": (lambda **o: nss.mb_layer_norm(x, w, b, **o), norm),
        "mb_layer_norm_backward": (lambda **o: nss.mb_layer_norm_backward(dy, x, mean, rstd, w, **o), back),
        "mb_rotary": (lambda **o: nss.mb_rotary(q, k, pos, freq, (16,), **o), rot),
        "mb_rotary_backward": (lambda **o: nss.mb_rotary_backward(q, k, pos, freq, (16,), **o), rot),
        "mb_router": (lambda **o: nss.mb_router(logits, 2, **o), route),
        "mb_router_backward": (lambda **o: nss.mb_router_backward(one, None, logits, *r[:3], r.used, **o), dlogits),
    }


def test_given_results_count_as_modified(nss):
    for name, (call, out) in _given(nss).items():
        before = {n: t._version for n, t in out.items()}
        call(**out)
        assert all(t._version > before[n] for n, t in out.items()), name
        before = {n: t._version for n, t in out.items()}
        wrong = {n: t[..., :0] for n, t in out.items()}
        with pytest.raises(ValueError):
            call(**wrong)
        assert all(t._version == before[n] for n, t in out.items()), f"{name}: a refused call"
        if len(out) > 1:
            first = next(iter(out))
            call(**{first: out[first]})
            assert [t._version > before[n] for n, t in out.items()] == [n == first for n in out], name


def test_overwriting_what_a_backward_pass_needs_is_noticed(nss):
    q, k, pos, freq = rotary_inputs(4, 1, 5, 2, 1, 16, (8,), torch.float32)
    q.requires_grad_()
    loss = q.square().sum()                                  # saves q
    nss.mb_rotary(q.detach(), None, pos, freq, (8,), q_out=q.detach())
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
    x, w, b, _ = norm_inputs(5, 8, 32, torch.float32, torch.float32)
    x.requires_grad_()
    loss = x.square().sum()
    nss.mb_layer_norm(x.detach(), w, b, y=x.detach())
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()


def test_results_made_in_inference_mode(nss):
    x, w, b, _ = norm_inputs(6, 8, 32, torch.float32, torch.float32)
    want = nss.mb_layer_norm(x, w, b)[0]
    with torch.inference_mode():
        y = torch.empty_like(x)
        same_bits(nss.mb_layer_norm(x, w, b, y=y)[0], want, "in inference mode")
    y.untyped_storage()                                      # an inference tensor has no version to move
    same_bits(nss.mb_layer_norm(x, w, b, y=y)[0], want, "afterwards")


def test_negated_views_are_refused(nss):
    """The imaginary part of a conjugate is a view whose memory holds the negated values: reading it as it lies would
    turn the wrong way."""
    q, _, pos, freq = rotary_inputs(7, 1, 6, 2, 1, 16, (8,), torch.float32)
    lazy = torch.complex(pos.float(), pos.float()).conj().imag
    assert lazy.is_neg() and torch.equal(lazy, -pos.float())
    for call in (nss.mb_rotary, nss.mb_rotary_backward):
        with pytest.raises(ValueError, match="resolve_neg"):
            call(q, None, lazy, freq, (8,))
        same_bits(call(q, None, lazy.resolve_neg(), freq, (8,))[0], call(q, None, -pos.float(), freq, (8,))[0], "resolved")
    x = torch.complex(q, q).conj().imag[..., :1]              # one element per row: any stride would do
    with pytest.raises(ValueError, match="resolve_neg"):
        nss.mb_layer_norm(x)
