"""The operators of a block between its matrix products: layer norm, rotary positions, expert routing.

Each function has the name of the C entry point it calls (include/muonbank.h gives the
formulas), takes CUDA tensors and enqueues the work on the current CUDA stream, or on
`stream`.  Results are new tensors unless the caller passes them; a given result may be the
input that it replaces.  Every operator has its gradient as a call of its own;
`newton_schulz_stacked_gb300.autograd` joins the pairs for torch's autograd.

Tensors may be strided in all but their last dimension; a tensor that is not laid out so, or
has another shape, type or device than the call's others, is refused with ValueError.  With
`stream`, new tensors belong to that stream and the given ones are marked as used on it; the
caller orders it after the stream that made them.
"""
from __future__ import annotations

import ctypes
import functools
import struct
from typing import NamedTuple, Optional, Sequence

import torch

from . import _binding as _b

_TYPES = {torch.float32: _b.MB_F32, torch.bfloat16: _b.MB_BF16, torch.float16: _b.MB_F16}
_POSITIONS = {torch.int32: _b.MB_I32, torch.int64: _b.MB_I64, torch.float32: _b.MB_F32}
_DESC = struct.Struct("@PPqqqqqqqPPqqqqqqqiiqqiiPqqqiiiiiiP")
assert _DESC.size == ctypes.sizeof(_b.MbRotaryDesc)


class RouterOutput(NamedTuple):
    """index int32 and gate fp32 [tokens, top_k]; counts int32 [experts]; loss fp32 [1]; used int32 [1]."""
    index: torch.Tensor
    gate: torch.Tensor
    counts: torch.Tensor
    loss: torch.Tensor
    used: torch.Tensor


def _cuda(t: torch.Tensor, what: str) -> torch.device:
    if not t.is_cuda:
        raise ValueError(f"{what} must be a CUDA tensor")
    return t.device


def _elsewhere(device, stream) -> bool:
    """Whether the call has to move to another stream or device first."""
    return stream is not None or torch.cuda.current_device() != device.index


def _moved(call, device, stream, tensors, args, kwargs):
    """The call with `device` current and on `stream`, with the tensors marked as used there."""
    with torch.cuda.device(device):
        if stream is None:
            return call(*args, **kwargs)
        if not isinstance(stream, torch.cuda.Stream):
            stream = torch.cuda.ExternalStream(stream, device) if stream else torch.cuda.default_stream(device)
        for t in tensors:
            if t is not None:
                t.record_stream(stream)
        with torch.cuda.stream(stream):
            return call(*args, **kwargs)


def _stream(device) -> int:
    return torch.cuda.current_stream(device).cuda_stream


def _type(t: torch.Tensor, what: str) -> int:
    try:
        return _TYPES[t.dtype]
    except KeyError:
        raise ValueError(f"{what} has dtype {t.dtype}, expected float32, bfloat16 or float16") from None


def _like(t: torch.Tensor, what: str, shape, dtype, device):
    if t.shape != shape or t.dtype != dtype or t.device != device:
        raise ValueError(f"{what} is {tuple(t.shape)} {t.dtype} on {t.device}, expected {tuple(shape)} {dtype} on {device}")


def _dense(t: Optional[torch.Tensor], what: str, shape, dtype, device) -> Optional[int]:
    """Address of a contiguous tensor of this shape and type (None: no tensor)."""
    if t is None:
        return None
    _like(t, what, shape, dtype, device)
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")
    return t.data_ptr()


def _row_stride(t: torch.Tensor, what: str) -> int:
    """Elements from row to row of t taken as [rows, t.shape[-1]]."""
    if t.is_contiguous():
        return t.shape[-1]
    if t.shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"{what} must be contiguous in its last dimension")
    stride, rows = None, 1          # dimensions of one element do not matter; the others must fold into one
    for n, s in zip(reversed(t.shape[:-1]), reversed(t.stride()[:-1])):
        if n == 1:
            continue
        if stride is None:
            stride = s
        elif s != stride * rows:
            raise ValueError(f"the rows of {what} must be evenly spaced")
        rows *= n
    return t.shape[-1] if stride is None else stride


@functools.lru_cache(maxsize=1024)
def _workspace_bytes(query: str, rows: int, cols: int) -> int:
    out = ctypes.c_size_t(0)
    _b.check(query, getattr(_b.load(), query)(rows, cols, ctypes.byref(out)))
    return out.value


def _workspace(query: str, rows: int, cols: int, workspace: Optional[torch.Tensor], device) -> torch.Tensor:
    need = _workspace_bytes(query, rows, cols)
    if workspace is None:
        return torch.empty(need, dtype=torch.uint8, device=device)
    if workspace.device != device or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on {device}")
    if workspace.numel() * workspace.element_size() < need:
        raise ValueError(f"workspace holds {workspace.numel() * workspace.element_size()} bytes, needs {need}")
    return workspace


# ---------------------------------------------------------------- layer norm

def _norm_shape(x: torch.Tensor, weight, device):
    if x.dim() < 1:
        raise ValueError("x must have at least one dimension")
    cols = x.shape[-1]
    if cols == 0:
        raise ValueError("x has rows of no elements")
    rows = x.numel() // cols
    wtype = _TYPES.get(weight.dtype) if weight is not None else _b.MB_F32
    if weight is not None and weight.dtype not in (x.dtype, torch.float32):
        raise ValueError(f"weight has dtype {weight.dtype}, expected {x.dtype} or float32")
    return rows, cols, wtype


def mb_layer_norm(x, weight=None, bias=None, eps: float = 1e-5, y=None, mean=None, rstd=None, stream=None):
    """Layer norm over the last dimension of x: (y, mean, rstd).

    weight and bias are [cols], in x's type or both in float32; mean and rstd are float32, one
    value per row, for mb_layer_norm_backward.
    """
    device = _cuda(x, "x")
    if _elsewhere(device, stream):
        return _moved(mb_layer_norm, device, stream, (x, weight, bias, y, mean, rstd), (x, weight, bias, eps, y, mean, rstd), {})
    kind = _type(x, "x")
    rows, cols, wtype = _norm_shape(x, weight if weight is not None else bias, device)
    wdtype = None if weight is None and bias is None else (weight if weight is not None else bias).dtype
    w = _dense(weight, "weight", (cols,), wdtype, device)
    b = _dense(bias, "bias", (cols,), wdtype, device)
    lead = x.shape[:-1]
    if y is None:
        y = torch.empty(x.shape, dtype=x.dtype, device=device)
    else:
        _like(y, "y", x.shape, x.dtype, device)
    if mean is None:
        mean = torch.empty(lead, dtype=torch.float32, device=device)
    if rstd is None:
        rstd = torch.empty(lead, dtype=torch.float32, device=device)
    st = _b.load().mb_layer_norm(
        x.data_ptr(), _row_stride(x, "x"), kind, w, b, wtype, y.data_ptr(), _row_stride(y, "y"),
        _dense(mean, "mean", lead, torch.float32, device), _dense(rstd, "rstd", lead, torch.float32, device), rows, cols,
        eps, _stream(device))
    if st:
        _b.check("mb_layer_norm", st)
    return y, mean, rstd


def mb_layer_norm_backward(dy, x, mean, rstd, weight=None, bias: bool = True, dx=None, dweight=None, dbias=None,
                           workspace=None, stream=None):
    """Gradients of mb_layer_norm: (dx, dweight, dbias).

    mean and rstd are the forward call's.  With a weight, dweight and (unless bias is False)
    dbias come in the weight's type; without one they are None.
    """
    device = _cuda(x, "x")
    if _elsewhere(device, stream):
        return _moved(mb_layer_norm_backward, device, stream,
                      (dy, x, mean, rstd, weight, dx, dweight, dbias, workspace),
                      (dy, x, mean, rstd, weight, bias, dx, dweight, dbias, workspace), {})
    kind = _type(x, "x")
    rows, cols, wtype = _norm_shape(x, weight, device)
    _like(dy, "dy", x.shape, x.dtype, device)
    lead = x.shape[:-1]
    if dx is None:
        dx = torch.empty(x.shape, dtype=x.dtype, device=device)
    else:
        _like(dx, "dx", x.shape, x.dtype, device)
    w = dw = db = ws = None
    nbytes = 0
    if weight is not None:
        w = _dense(weight, "weight", (cols,), weight.dtype, device)
        if dweight is None:
            dweight = torch.empty(cols, dtype=weight.dtype, device=device)
        if dbias is None and bias:
            dbias = torch.empty(cols, dtype=weight.dtype, device=device)
        dw = _dense(dweight, "dweight", (cols,), weight.dtype, device)
        db = _dense(dbias, "dbias", (cols,), weight.dtype, device)
        workspace = _workspace("mb_layer_norm_workspace_bytes", rows, cols, workspace, device)
        ws, nbytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    elif dweight is not None or dbias is not None:
        raise ValueError("dweight and dbias need a weight")
    st = _b.load().mb_layer_norm_backward(
        dy.data_ptr(), _row_stride(dy, "dy"), x.data_ptr(), _row_stride(x, "x"), kind, w, wtype,
        _dense(mean, "mean", lead, torch.float32, device), _dense(rstd, "rstd", lead, torch.float32, device),
        dx.data_ptr(), _row_stride(dx, "dx"), dw, db, rows, cols, ws, nbytes, _stream(device))
    if st:
        _b.check("mb_layer_norm_backward", st)
    return dx, dweight, dbias


# ---------------------------------------------------------------- rotary positions

def _heads(t: torch.Tensor, what: str, shape4) -> tuple:
    """(strides of batch, token, head); the elements of a head are contiguous."""
    if shape4[3] > 1 and t.stride(-1) != 1:
        raise ValueError(f"{what} must be contiguous in its last dimension")
    s = t.stride()
    return s[:3] if len(s) == 4 else (0, s[0], s[1])


def _rotary(name, q, k, positions, inv_freq, sections, interleaved, q_out, k_out, stream):
    device = _cuda(q, "q")
    if _elsewhere(device, stream):
        return _moved(_rotary, device, stream, (q, k, positions, inv_freq, q_out, k_out),
                      (name, q, k, positions, inv_freq, sections, interleaved, q_out, k_out, None), {})
    kind = _type(q, "q")
    if q.dim() not in (3, 4):
        raise ValueError("q must be [batch, tokens, heads, dim] or [tokens, heads, dim]")
    shape = tuple(q.shape) if q.dim() == 4 else (1,) + tuple(q.shape)
    batch, tokens, heads, dim = shape
    if q_out is None:
        q_out = torch.empty(q.shape, dtype=q.dtype, device=device)
    else:
        _like(q_out, "q_out", q.shape, q.dtype, device)
    qs, qd = _heads(q, "q", shape), _heads(q_out, "q_out", shape)
    kp = kd_ptr = kv_heads = 0
    ks = kd = (0, 0, 0)
    if k is not None:
        kv_heads = k.shape[-2] if k.dim() == q.dim() else 0
        _like(k, "k", q.shape[:-2] + (kv_heads, dim), q.dtype, device)
        if k_out is None:
            k_out = torch.empty(k.shape, dtype=k.dtype, device=device)
        else:
            _like(k_out, "k_out", k.shape, k.dtype, device)
        ks, kd = _heads(k, "k", shape), _heads(k_out, "k_out", shape)
        kp, kd_ptr = k.data_ptr(), k_out.data_ptr()
    elif k_out is not None:
        raise ValueError("k_out needs a k")
    axes = len(sections)
    if not 1 <= axes <= _b.MB_ROTARY_MAX_AXES:
        raise ValueError(f"sections has {axes} axes, expected 1 to {_b.MB_ROTARY_MAX_AXES}")
    pairs = inv_freq.numel()
    if sum(sections) != pairs:
        raise ValueError(f"sections add up to {sum(sections)} pairs, inv_freq has {pairs}")
    freq = _dense(inv_freq, "inv_freq", (pairs,), torch.float32, device)
    if positions.dtype not in _POSITIONS:
        raise ValueError(f"positions has dtype {positions.dtype}, expected int32, int64 or float32")
    ps = positions.stride()
    if positions.dim() == 2:             # the same positions in every sequence
        _like(positions, "positions", (axes, tokens), positions.dtype, device)
        ps = (ps[0], 0, ps[1])
    else:
        _like(positions, "positions", (axes, batch, tokens), positions.dtype, device)
    sec = tuple(sections) + (0,) * (_b.MB_ROTARY_MAX_AXES - axes)
    try:
        desc = _DESC.pack(q.data_ptr(), q_out.data_ptr(), heads, *qs, *qd, kp, kd_ptr, kv_heads, *ks, *kd, kind,
                          bool(interleaved), batch, tokens, dim, pairs, positions.data_ptr(), *ps,
                          _POSITIONS[positions.dtype], axes, *sec, freq)
    except struct.error as e:
        raise ValueError(f"{name}: a size or section out of range ({e})") from None
    st = getattr(_b.load(), name)(desc, _stream(device))
    if st:
        _b.check(name, st)
    return q_out, k_out


def mb_rotary(q, k, positions, inv_freq, sections: Sequence[int], interleaved: bool = False, q_out=None, k_out=None,
              stream=None):
    """Rotary positions on q and k (k may be None): (q_out, k_out).

    q is [batch, tokens, heads, dim] (or without the batch), k the same with its own number of
    heads.  positions is [axes, batch, tokens], or [axes, tokens] for all sequences, in int32,
    int64 or float32; inv_freq is float32 [pairs], and `sections` says how many of the pairs, in
    order, each axis turns.  Pairs are (i, i + pairs), or (2i, 2i + 1) if interleaved; the
    elements of a head past 2 * pairs are copied.
    """
    return _rotary("mb_rotary", q, k, positions, inv_freq, sections, interleaved, q_out, k_out, stream)


def mb_rotary_backward(dq, dk, positions, inv_freq, sections: Sequence[int], interleaved: bool = False, q_out=None,
                       k_out=None, stream=None):
    """Gradients of mb_rotary with respect to q and k from those of its results (dk may be None)."""
    return _rotary("mb_rotary_backward", dq, dk, positions, inv_freq, sections, interleaved, q_out, k_out, stream)


# ---------------------------------------------------------------- router

def _router_shape(logits, top_k):
    if logits.dim() != 2:
        raise ValueError("logits must be [tokens, experts]")
    return logits.shape[0], logits.shape[1], int(top_k)


def _valid(valid, tokens, device) -> Optional[int]:
    if valid is None:
        return None
    if valid.dtype not in (torch.bool, torch.uint8):
        raise ValueError(f"valid has dtype {valid.dtype}, expected bool or uint8")
    return _dense(valid, "valid", (tokens,), valid.dtype, device)


def mb_router(logits, top_k: int, valid=None, normalize: bool = False, index=None, gate=None, counts=None, loss=None,
              used=None, workspace=None, stream=None) -> RouterOutput:
    """Top-k routing of tokens over experts: RouterOutput(index, gate, counts, loss, used).

    valid (bool or uint8 [tokens]) leaves tokens out, -inf among the logits closes an expert
    for a token; a place without an expert has index -1 and gate 0.  With normalize a token's
    gates add up to 1.  `loss` is the balance loss (1 when balanced), `used` the number of
    tokens that count.
    """
    device = _cuda(logits, "logits")
    if _elsewhere(device, stream):
        return _moved(mb_router, device, stream, (logits, valid, index, gate, counts, loss, used, workspace),
                      (logits, top_k, valid, normalize, index, gate, counts, loss, used, workspace), {})
    kind = _type(logits, "logits")
    tokens, experts, top_k = _router_shape(logits, top_k)
    ws = _workspace("mb_router_workspace_bytes", tokens, experts, workspace, device)
    chosen = (tokens, max(top_k, 0))
    if index is None:
        index = torch.empty(chosen, dtype=torch.int32, device=device)
    if gate is None:
        gate = torch.empty(chosen, dtype=torch.float32, device=device)
    if counts is None:
        counts = torch.empty(experts, dtype=torch.int32, device=device)
    if loss is None:
        loss = torch.empty(1, dtype=torch.float32, device=device)
    if used is None:
        used = torch.empty(1, dtype=torch.int32, device=device)
    st = _b.load().mb_router(
        logits.data_ptr(), _row_stride(logits, "logits"), kind, _valid(valid, tokens, device), tokens, experts, top_k,
        bool(normalize), _dense(index, "index", chosen, torch.int32, device),
        _dense(gate, "gate", chosen, torch.float32, device), _dense(counts, "counts", (experts,), torch.int32, device),
        _dense(loss, "loss", (1,), torch.float32, device), _dense(used, "used", (1,), torch.int32, device),
        ws.data_ptr(), ws.numel() * ws.element_size(), _stream(device))
    if st:
        _b.check("mb_router", st)
    return RouterOutput(index, gate, counts, loss, used)


def mb_router_backward(dloss, dgate, logits, index, gate, counts, used, valid=None, normalize: bool = False, dlogits=None,
                       stream=None):
    """Gradient of mb_router's logits from those of its loss (float32 [1]) and gates (float32
    [tokens, top_k]); either may be None.  index, gate, counts and used are the forward call's."""
    device = _cuda(logits, "logits")
    if _elsewhere(device, stream):
        return _moved(mb_router_backward, device, stream,
                      (dloss, dgate, logits, index, gate, counts, used, valid, dlogits),
                      (dloss, dgate, logits, index, gate, counts, used, valid, normalize, dlogits), {})
    kind = _type(logits, "logits")
    if index.dim() != 2:
        raise ValueError("index must be [tokens, top_k]")
    tokens, experts, top_k = _router_shape(logits, index.shape[1])
    chosen = (tokens, top_k)
    if dlogits is None:
        dlogits = torch.empty((tokens, experts), dtype=logits.dtype, device=device)
    else:
        _like(dlogits, "dlogits", logits.shape, logits.dtype, device)
    st = _b.load().mb_router_backward(
        _dense(dloss, "dloss", (1,), torch.float32, device), _dense(dgate, "dgate", chosen, torch.float32, device),
        logits.data_ptr(), _row_stride(logits, "logits"), kind, _valid(valid, tokens, device), tokens, experts, top_k,
        bool(normalize), _dense(index, "index", chosen, torch.int32, device),
        _dense(gate, "gate", chosen, torch.float32, device), _dense(counts, "counts", (experts,), torch.int32, device),
        _dense(used, "used", (1,), torch.int32, device), dlogits.data_ptr(), _row_stride(dlogits, "dlogits"),
        _stream(device))
    if st:
        _b.check("mb_router_backward", st)
    return dlogits
