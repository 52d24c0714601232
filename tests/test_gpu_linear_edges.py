"""The products at the edges of what a call may ask of them: values, layouts, sizes on both sides of the rules that choose a
kernel.  Tolerances are those of test_gpu_linear.py, whose plain forms in 64 bits these tests take."""
import math

import pytest
import torch

from test_gpu_linear import ACTS, _add, _gen, _near, _rows, _slope, nss  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("rows", [4, 300])
def test_slopes_of_large_finite_values(nss, act, rows):
    """Values whose powers pass fp32: the slope is finite where the formula's is."""
    g, t, cols, out = _gen(41), torch.bfloat16, 64, 64
    x, w, dy, z = _rows(rows, cols, t, g), _rows(out, cols, t, g, std=cols ** -0.5), _rows(rows, out, t, g), _rows(rows, out, t, g)
    sizes = [15.0, 16.0, 17.0, 1e3, 1e6, 1e12, 1e14, 1e18, 1e20, 1e30, 1e38, 3.3e38]
    z[1, :len(sizes)] = torch.tensor(sizes, device="cuda")
    z[2, :len(sizes)] = -torch.tensor(sizes, device="cuda")
    if act == "relu2":                           # a slope of 2 z: dz of these is infinite in earnest
        z[1:3, sizes.index(1e30):len(sizes)] = 1.0
        dy[1:3] *= 2.0 ** -100
    dx, dw, db = nss.mb_linear_backward(dy, x, w, z, act, bias=True)
    want = dy.double() * (torch.ones_like(z) if act == "none" else _wide_slope(z.double(), act))
    assert dx.isfinite().all() and dw.isfinite().all() and db.isfinite().all()
    _near(db, want.sum(0), (_add(rows) + 2.0 ** -18) * want.abs().sum(0))
    if act != "none":                            # an infinity stays one that shows
        z[3, 5] = math.inf
        dx, _, _ = nss.mb_linear_backward(dy, x, w, z, act)
        shown = not dx[3].isfinite().all()
        assert shown == (act != "relu") and dx[:3].isfinite().all()


def _wide_slope(z, act):
    """The derivative, by its limits where the powers of z pass 64 bits' range too."""
    far = z.abs() > 1e3
    near = _slope(torch.where(far, 1.0, z), act)
    return torch.where(far, 2 * z.clamp(min=0) if act == "relu2" else (z > 0).double(), near)
