"""The operators of a block: products with bias, activation and residual, layer norm, rotary positions, expert routing.

Each function has the name of the C entry point it calls (include/muonbank.h gives the
formulas), takes CUDA tensors and enqueues the work on the current CUDA stream, or on
`stream`.  Results are new tensors unless the caller passes them; a given result may be the
input that it replaces, and counts as modified in place.  New tensors of one call may share an
allocation (mean and rstd; index and gate; counts, loss and used).  Every operator has its gradient
as a call of its own; autograd does not record these calls, but
`newton_schulz_stacked_gb300.autograd` joins the pairs for it.

Tensors may be strided in all but their last dimension (a norm's rows evenly spaced); a tensor that is not laid out so, or
has another shape, type or device than the call's others, is refused with ValueError, and what
the library refuses raises MuonBankError.  With `stream` (a torch stream or its handle), new
tensors belong to that stream and the given ones are marked as used on it; the caller orders
it after the stream that made them.

The checks, the new tensors and the C call are one native call (csrc/mb_torch.cpp).
"""
from __future__ import annotations

import importlib
import os
from typing import NamedTuple, Sequence

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
_native = None


def load_binding():
    """The native binding (raises if it has not been built)."""
    global _native
    if _native is None:
        if not os.path.exists(os.path.join(HERE, "_blocks.so")):
            raise RuntimeError("_blocks.so is missing: build it with __graft_entry__.build() or "
                               "python -m newton_schulz_stacked_gb300.build")
        _native = importlib.import_module("newton_schulz_stacked_gb300._blocks")
    return _native


class RouterOutput(NamedTuple):
    """index int32 and gate fp32 [tokens, top_k]; counts int32 [experts]; loss fp32 [1]; used int32 [1]."""
    index: torch.Tensor
    gate: torch.Tensor
    counts: torch.Tensor
    loss: torch.Tensor
    used: torch.Tensor


def mb_layer_norm(x, weight=None, bias=None, eps: float = 1e-5, y=None, mean=None, rstd=None, stream=None):
    """Layer norm over the last dimension of x: (y, mean, rstd).

    weight and bias are [cols], in x's type or both in float32; mean and rstd are float32, one
    value per row, for mb_layer_norm_backward.
    """
    return (_native or load_binding()).mb_layer_norm(x, weight, bias, eps, y, mean, rstd, stream)


def mb_layer_norm_backward(dy, x, mean, rstd, weight=None, bias: bool = True, dx=None, dweight=None, dbias=None,
                           workspace=None, stream=None, weight_grad: bool = True):
    """Gradients of mb_layer_norm: (dx, dweight, dbias).

    mean and rstd are the forward call's.  With a weight, dweight (unless weight_grad is False) and
    dbias (unless bias is False) come in the weight's type; without one they are None, but a dbias
    that is passed, in x's type or float32, is written.  Without either the sums over the rows are
    left out, and with them a launch.
    """
    return (_native or load_binding()).mb_layer_norm_backward(dy, x, mean, rstd, weight, bias, dx, dweight, dbias,
                                                              workspace, stream, weight_grad)


def mb_rotary(q, k, positions, inv_freq, sections: Sequence[int], interleaved: bool = False, q_out=None, k_out=None,
              stream=None):
    """Rotary positions on q and k (k may be None): (q_out, k_out).

    q is [batch, tokens, heads, dim] (or without the batch), k the same with its own number of
    heads.  positions is [axes, batch, tokens], or [axes, tokens] for all sequences, in int32,
    int64 or float32; inv_freq is float32 [pairs], and `sections` says how many of the pairs, in
    order, each axis turns.  Pairs are (i, i + pairs), or (2i, 2i + 1) if interleaved; the
    elements of a head past 2 * pairs are copied.
    """
    return (_native or load_binding()).mb_rotary(q, k, positions, inv_freq, sections, interleaved, q_out, k_out, stream)


def mb_rotary_backward(dq, dk, positions, inv_freq, sections: Sequence[int], interleaved: bool = False, q_out=None,
                       k_out=None, stream=None):
    """Gradients of mb_rotary with respect to q and k from those of its results (dk may be None)."""
    return (_native or load_binding()).mb_rotary_backward(dq, dk, positions, inv_freq, sections, interleaved, q_out,
                                                          k_out, stream)


def mb_router(logits, top_k: int, valid=None, normalize: bool = False, index=None, gate=None, counts=None, loss=None,
              used=None, workspace=None, stream=None) -> RouterOutput:
    """Top-k routing of tokens over experts: RouterOutput(index, gate, counts, loss, used).

    valid (bool or uint8 [tokens]) leaves tokens out, -inf among the logits closes an expert
    for a token; a place without an expert has index -1 and gate 0.  With normalize a token's
    gates add up to 1.  `loss` is the balance loss (1 when balanced), `used` the number of
    tokens that count.
    """
    return tuple.__new__(RouterOutput, (_native or load_binding()).mb_router(
        logits, top_k, valid, normalize, index, gate, counts, loss, used, workspace, stream))


def mb_router_backward(dloss, dgate, logits, index, gate, counts, used, valid=None, normalize: bool = False, dlogits=None,
                       stream=None):
    """Gradient of mb_router's logits from those of its loss (float32 [1]) and gates (float32
    [tokens, top_k]); either may be None.  index, gate, counts and used are the forward call's."""
    return (_native or load_binding()).mb_router_backward(dloss, dgate, logits, index, gate, counts, used, valid, normalize,
                                                          dlogits, stream)


def mb_linear(x, weight, bias=None, residual=None, activation: str = "none", ends=None, keep: bool = False, y=None, z=None,
              workspace=None, stream=None):
    """act(x W^T + bias) + residual: (y, z), z = x W^T + bias if keep (for the backward pass), else None.

    x is [..., in] in bfloat16 or float16, weight [out, in], bias [out] in x's type or float32, residual
    [..., out].  With `ends`, int32 [groups], weight is a bank [groups, out, in] (and bias [groups, out]): the rows of x
    are consecutive groups, group g ending before row ends[g], such as tokens sorted by expert with
    ends = counts.cumsum(0, dtype=torch.int32); rows from the last end on get zeros.  The ends stay on the device.
    activation: "none", "relu", "relu2" (its square), "silu" or "gelu" (the tanh form).  A few rows (single tokens, up to
    512) take kernels of their own, without tiles, where those are the shorter way.  y may be the residual, with its
    strides; a result that shares memory with anything else of the call is refused.
    """
    return (_native or load_binding()).mb_linear(x, weight, bias, residual, activation, ends, keep, y, z, workspace, stream)


def mb_linear_backward(dy, x, weight, z=None, activation: str = "none", ends=None, input_grad: bool = True,
                       weight_grad: bool = True, bias: bool = False, dx=None, dweight=None, dbias=None, workspace=None,
                       stream=None):
    """Gradients of mb_linear: (dx, dweight, dbias), None for those that are not wanted (input_grad, weight_grad, bias).

    z is the forward call's (not needed without an activation).  x is read for dweight only, weight for dx only: either may be
    None where that gradient is not wanted.  dweight is laid out as the weight, the gradient of a bank as
    muon_multi_step takes it; dbias comes in x's type unless a float32 one is passed.  The residual's gradient is dy.  A result
    that shares memory with anything else of the call is refused.
    """
    return (_native or load_binding()).mb_linear_backward(dy, x, weight, z, activation, ends, input_grad, weight_grad, bias,
                                                          dx, dweight, dbias, workspace, stream)
