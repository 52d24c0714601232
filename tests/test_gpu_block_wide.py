"""Layer norm of rows of more than 8192 elements with more rows than the kernels have CTAs or slabs, so that every loop over
rows takes several turns (at most two CTAs per SM, 64 slabs for the weight's gradient)."""
import ctypes

import pytest
import torch

from test_gpu_blocks import (TYPES, U, Guarded, check_norm_forward, norm_backward_ref, norm_inputs, nss, rounding,   # noqa: F401
                             same_bits, within)

pytestmark = pytest.mark.gpu

ROWS = 700
SLABS = 64


def wide_param_bounds(dy, x, mean, rstd, wtype):
    """(dw, its bound, db, its bound): a thread adds one row in 64 (each term: the difference, its product with rstd, and the
    fused addition), 32 slices add two slabs each, and a warp's exchanges add the slices."""
    rows = x.shape[0]
    dyd = dy.double()
    h = (x.double() - mean.double()[:, None]) * rstd.double()[:, None]
    E = -(-rows // SLABS) + 2 + SLABS // 32 + 5 + 1
    dw, db = (dyd * h).sum(0), dyd.sum(0)
    return (dw, 1.01 * E * U * (dyd * h).abs().sum(0) + rounding(dw, wtype), db,
            1.01 * E * U * dyd.abs().sum(0) + rounding(db, wtype))


# 16-byte pieces and single elements; 16384 is the last width that the forward pass holds by single elements, 32768 by pieces
@pytest.mark.parametrize("cols", [8200, 8203, 16391, 32768, 33000, 33001])
@pytest.mark.parametrize("dtype,wtype", [("bf16", "f32"), ("bf16", "bf16"), ("f16", "f32"), ("f32", "f32")])
def test_wide_rows(nss, cols, dtype, wtype):
    x, w, b, dy = norm_inputs(cols, ROWS, cols, TYPES[dtype], TYPES[wtype])
    _, mean, rstd = check_norm_forward(nss, x, w, b)
    dx, dw, db = nss.mb_layer_norm_backward(dy, x, mean, rstd, w)
    torch.cuda.synchronize()
    ref, bound = norm_backward_ref(dy, x, mean, rstd, w)[:2]
    within(dx, ref, bound, "dx")
    rw, bw, rb, bb = wide_param_bounds(dy, x, mean, rstd, TYPES[wtype])
    within(dw, rw, bw, "dw")
    within(db, rb, bb, "db")
    # over its inputs, the same bits
    y = nss.mb_layer_norm(x, w, b)[0]
    over = x.clone()
    nss.mb_layer_norm(over, w, b, y=over)
    same_bits(over, y, "y over x")
    for over_x in (True, False):
        xx, dd = x.clone(), dy.clone()
        got = nss.mb_layer_norm_backward(dd, xx, mean, rstd, w, dx=xx if over_x else dd)
        for a, c, what in zip(got, (dx, dw, db), ("dx", "dw", "db")):
            same_bits(a, c, f"{what} over {'x' if over_x else 'dy'}")


@pytest.mark.parametrize("cols", [8200, 8203, 33000, 33001])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_bad_wide_rows_stay_alone(nss, cols, dtype):
    """A row that is not finite leaves nothing behind in what its CTA shares with the rows after it."""
    x, w, b, dy = norm_inputs(cols + 1, ROWS, cols, TYPES[dtype], torch.float32)
    y, mean, rstd = nss.mb_layer_norm(x, w, b)
    dx = nss.mb_layer_norm_backward(dy, x, mean, rstd, w)[0]
    bad = torch.zeros(ROWS, dtype=torch.bool, device="cuda")
    bad[[0, 151, 303, 304, 607]] = True
    dirty = x.clone()
    dirty[bad, cols // 2] = float("nan")
    got = nss.mb_layer_norm(dirty, w, b)
    assert torch.isnan(got[0][bad]).all()
    for a, c in zip(got, (y, mean, rstd)):
        same_bits(a[~bad], c[~bad], "beside a bad row")
    back = nss.mb_layer_norm_backward(dy, dirty, got[1], got[2], w)
    assert torch.isnan(back[0][bad]).all() and torch.isnan(back[1]).all()
    same_bits(back[0][~bad], dx[~bad], "dx beside a bad row")


@pytest.mark.parametrize("rows", [1, 63, 64, 65, 300, ROWS])
@pytest.mark.parametrize("cols", [96, 777, 2048, 2051, 8192, 8200, 8203])
def test_workspace_of_the_needed_size(nss, rows, cols):
    """A given workspace of exactly the bytes asked for is enough, nothing beyond it is written, and its contents do not matter."""
    x, w, b, dy = norm_inputs(rows + cols, rows, cols, torch.bfloat16, torch.float32)
    _, mean, rstd = nss.mb_layer_norm(x, w, b)
    want = nss.mb_layer_norm_backward(dy, x, mean, rstd, w)
    need = ctypes.c_size_t()
    from newton_schulz_stacked_gb300 import _binding as B
    B.check("mb_layer_norm_workspace_bytes", B.load().mb_layer_norm_workspace_bytes(rows, cols, ctypes.byref(need)))
    room = torch.full((need.value + 4096,), 0xFF, device="cuda", dtype=torch.uint8)      # NaN, read as fp32
    got = nss.mb_layer_norm_backward(dy, x, mean, rstd, w, workspace=room[:need.value])
    for a, c, what in zip(got, want, ("dx", "dw", "db")):
        same_bits(a, c, what)
    assert bool((room[need.value:] == 0xFF).all()), "wrote past the workspace"
    dx = Guarded((rows, cols), torch.bfloat16, 8, 0)
    nss.mb_layer_norm_backward(dy, x, mean, rstd, w, dx=dx.t, workspace=room)            # and a larger one
    dx.check("dx")


@pytest.mark.parametrize("tokens,experts,k", [(5000, 64, 4), (300, 1000, 8), (100, 512, 2)])
def test_router_workspace_of_the_needed_size(nss, tokens, experts, k):
    logits = torch.randn(tokens, experts, device="cuda", generator=torch.Generator(device="cuda").manual_seed(tokens))
    want = nss.mb_router(logits, k)
    need = ctypes.c_size_t()
    from newton_schulz_stacked_gb300 import _binding as B
    B.check("mb_router_workspace_bytes", B.load().mb_router_workspace_bytes(tokens, experts, ctypes.byref(need)))
    assert need.value > 0
    room = torch.full((need.value + 4096,), 0xFF, device="cuda", dtype=torch.uint8)
    for a, c, what in zip(nss.mb_router(logits, k, workspace=room[:need.value]), want, want._fields):
        same_bits(a, c, what)
    assert bool((room[need.value:] == 0xFF).all()), "wrote past the workspace"
