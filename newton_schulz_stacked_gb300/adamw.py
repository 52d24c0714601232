"""AdamW over the tensors that are in no bank: embeddings, heads, norms, biases.

adamw_multi_step steps a whole list in one launch; include/muonbank.h gives the formulas and the 8-bit
moments' format.  The tensors are the caller's and are updated in place; they must be contiguous, and what a
call writes may not overlap anything else of it (gradients, which are only read, may share memory with one
another).  What is laid out otherwise, or has another size, type or device, is refused with ValueError before
anything is stepped; what the library refuses raises MuonBankError.
"""
from __future__ import annotations

from typing import NamedTuple, Optional, Sequence

import torch

from . import blocks as _k

BLOCK = 256     # consecutive elements that share a scale of 8-bit moments


class AdamState(NamedTuple):
    """One tensor of a step.

    param float32, bfloat16 or float16; grad of its shape in any of these.  exp_avg and exp_avg_sq have as many
    elements, in float32, or both in float8_e4m3fn with avg_scale and sq_scale, float32 of one value per 256
    elements (then exp_avg * avg_scale is the first moment, exp_avg_sq * sq_scale the root of the second).
    mantissa (int16 or uint16 bits) makes a bfloat16 param the high half of an fp32 weight, as a bank's is.
    lr_mul and wd_mul multiply the call's lr and wd.
    """
    param: torch.Tensor
    grad: torch.Tensor
    exp_avg: torch.Tensor
    exp_avg_sq: torch.Tensor
    mantissa: Optional[torch.Tensor] = None
    avg_scale: Optional[torch.Tensor] = None
    sq_scale: Optional[torch.Tensor] = None
    lr_mul: float = 1.0
    wd_mul: float = 1.0


def adamw_state(param, grad=None, mantissa=None, bits: int = 32, lr_mul: float = 1.0, wd_mul: float = 1.0) -> AdamState:
    """The state of a tensor before its first step, with moments in 32 or 8 bits.  Each step's gradient is put in with
    state._replace(grad=...)."""
    if bits not in (8, 32):
        raise ValueError(f"bits is {bits}, expected 8 or 32")
    param = param.detach()
    like = {"device": param.device, "dtype": torch.float32 if bits == 32 else torch.float8_e4m3fn}
    avg, sq = torch.zeros(param.shape, **like), torch.zeros(param.shape, **like)
    scales = (None, None)
    if bits == 8:
        scales = tuple(torch.zeros(-(-param.numel() // BLOCK), device=param.device) for _ in range(2))
    return AdamState(param, grad, avg, sq, mantissa, *scales, lr_mul, wd_mul)


def adamw_multi_step(tensors: Sequence[AdamState], lr: float, wd: float, beta1: float = 0.9, beta2: float = 0.95,
                     eps: float = 1e-8, step: int = 1, grad_scale=None, seed: Optional[int] = None, stream=None) -> None:
    """One AdamW step of every tensor of the list, in place.

    step counts from 1.  grad_scale, a CUDA float32 tensor of one value (a scalar, or of shape [1]), multiplies every
    gradient (a clipping factor).  With a seed (0 to 2^32 - 1) 8-bit moments are rounded at random, the same way for the same seed, step
    and place in the list; without one, to the nearest.
    """
    (_k._native or _k.load_binding()).adamw_multi_step(tensors, lr, wd, beta1, beta2, eps, step, grad_scale, seed, stream)


def adamw_multi_step_dev(tensors: Sequence[AdamState], scalars, grad_scale=None, seed: Optional[int] = None, workspace=None,
                         stream=None):
    """adamw_multi_step with (lr, wd, beta1, beta2, eps, step) read from `scalars`, a CUDA float64 tensor of six values,
    when the step runs: a captured CUDA graph replays with what it then holds.  Returns the workspace."""
    return (_k._native or _k.load_binding()).adamw_multi_step_dev(tensors, scalars, grad_scale, seed, workspace, stream)
