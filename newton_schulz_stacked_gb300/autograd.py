"""The block operators under torch's autograd: each forward call joined with its backward call.

rotary is linear in q and k and can be differentiated any number of times.  layer_norm and route
have first derivatives only: differentiating their gradients (of create_graph=True) raises
RuntimeError.
"""
from __future__ import annotations

from typing import NamedTuple, Sequence

import torch

from . import blocks as _k


class Routing(NamedTuple):
    """index int32 and gate fp32 [tokens, top_k], counts int32 [experts], loss fp32 scalar."""
    index: torch.Tensor
    gate: torch.Tensor
    counts: torch.Tensor
    loss: torch.Tensor


def _readable(g: torch.Tensor) -> torch.Tensor:
    """Autograd may hand over an expanded gradient (of a sum, say) or a negated view (through a conjugate): its
    elements are laid out first."""
    g = g.resolve_neg()
    return g if g.shape[-1] == 1 or g.stride(-1) == 1 else g.contiguous()


class _FirstOnly(torch.autograd.Function):
    """A gradient that has none itself.  Its inputs tie it into the graph, so that the gradient is not
    taken for a constant: a second derivative that needs it raises."""

    @staticmethod
    def forward(ctx, name, call, *inputs):
        ctx.name = name
        return call(*inputs)

    @staticmethod
    def backward(ctx, *_):
        raise RuntimeError(f"{ctx.name} has no second derivative")


def _first_only(name, call, *inputs):
    """call(*inputs); under create_graph=True, as a step of the graph."""
    return _FirstOnly.apply(name, call, *inputs) if torch.is_grad_enabled() else call(*inputs)


class _LayerNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, eps):
        y, mean, rstd = _k.mb_layer_norm(x, weight, bias, eps)
        ctx.save_for_backward(x, weight, mean, rstd)
        return y

    @staticmethod
    def backward(ctx, dy):
        x, weight, mean, rstd = ctx.saved_tensors
        dy = dy.resolve_neg().contiguous()
        _, weight_grad, bias_grad, _ = ctx.needs_input_grad   # not of frozen parameters
        dx, dweight, dbias = _first_only(
            "layer_norm", lambda *t: _k.mb_layer_norm_backward(*t, bias=bias_grad, weight_grad=weight_grad), dy, x, mean,
            rstd, weight)
        return dx, dweight, dbias, None


def layer_norm(x, weight=None, bias=None, eps: float = 1e-5) -> torch.Tensor:
    """Layer norm over the last dimension, differentiable in x, weight and bias."""
    if weight is None and bias is not None:
        raise ValueError("a bias needs a weight")
    return _LayerNorm.apply(x, weight, bias, eps)


class _Rotary(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, positions, inv_freq, sections, interleaved, back):
        ctx.save_for_backward(positions, inv_freq)
        ctx.args = sections, interleaved
        ctx.back = back
        ctx.set_materialize_grads(False)
        return (_k.mb_rotary_backward if back else _k.mb_rotary)(q, k, positions, inv_freq, sections, interleaved)

    @staticmethod
    def backward(ctx, dq, dk):
        def turn_back(a, b):
            b = None if b is None else _readable(b)
            return _Rotary.apply(_readable(a), b, *ctx.saved_tensors, *ctx.args, not ctx.back)

        if dq is not None:
            dq, dk = turn_back(dq, dk)
        elif dk is not None:
            dk, _ = turn_back(dk, None)
        return dq, dk, None, None, None, None, None


def rotary(q, k, positions, inv_freq, sections: Sequence[int], interleaved: bool = False):
    """mb_rotary, differentiable in q and k (k may be None): (q_out, k_out).  positions and inv_freq have no
    gradient: one that requires it is refused."""
    for name, t in (("positions", positions), ("inv_freq", inv_freq)):
        if t.requires_grad and torch.is_grad_enabled():
            raise ValueError(f"{name} requires a gradient, which rotary does not have: pass {name}.detach()")
    return _Rotary.apply(q, k, positions, inv_freq, tuple(sections), interleaved, False)


class _Route(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, top_k, valid, normalize):
        out = _k.mb_router(logits, top_k, valid, normalize)
        ctx.save_for_backward(logits, valid, out.index, out.gate, out.counts, out.used)
        ctx.normalize = normalize
        ctx.mark_non_differentiable(out.index, out.counts)
        ctx.set_materialize_grads(False)
        return out.index, out.gate, out.counts, out.loss.reshape(())

    @staticmethod
    def backward(ctx, _index, dgate, _counts, dloss):
        if dgate is None and dloss is None:
            return None, None, None, None
        logits, valid, index, gate, counts, used = ctx.saved_tensors
        dlogits = _first_only(
            "route", lambda *t: _k.mb_router_backward(*t, normalize=ctx.normalize), None if dloss is None else dloss.resolve_neg().reshape(1),
            None if dgate is None else dgate.resolve_neg().contiguous(), logits, index, gate, counts, used, valid)
        return dlogits, None, None, None


def route(logits, top_k: int, valid=None, normalize: bool = False) -> Routing:
    """mb_router, differentiable in the logits through the gates and the balance loss."""
    return Routing(*_Route.apply(logits, top_k, valid, normalize))
