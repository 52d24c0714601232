"""Routing of tokens whose logits are NaN, alone and beside closed experts, with all experts chosen or nearly so.

The lanes of a token hold more places than there are experts here, so a choice made by the places' keys
alone would meet those past the last expert.
"""
import pytest
import torch

from test_gpu_blocks import Guarded, TYPES, check_router, gen, nss, randn      # noqa: F401  (nss is a fixture)

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("experts,k", [(1, 1), (2, 2), (3, 3), (5, 5), (6, 6), (7, 7), (7, 6), (8, 8), (9, 9), (12, 12), (15, 14),
                                       (16, 16), (20, 20), (24, 24), (31, 31), (32, 32), (33, 32), (60, 32), (100, 5), (250, 32)])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_router_nan_beside_closed_experts(nss, experts, k, dtype):
    g, t = gen(experts), 70
    box = Guarded((t, experts), TYPES[dtype], 8, 0)
    logits = randn(g, t, experts)
    some = torch.rand((t, experts), generator=g, device="cuda") < 0.4
    some[:, 0] |= ~some.any(1)
    kind = torch.arange(t, device="cuda") % 7
    logits[kind == 1] = NAN                                              # nothing but NaN
    logits[kind == 2] = torch.where(some, NAN, -INF)[kind == 2]          # NaN beside closed experts
    logits[kind == 3] = torch.where(some, logits, NAN)[kind == 3]        # beside ordinary ones
    logits[kind == 4] = torch.where(some, logits, -INF)[kind == 4]       # closed experts beside ordinary ones
    logits[kind == 5] = -INF
    logits[t - 1] = NAN                                                  # the last row of the buffer
    kind[t - 1] = 1
    box.t.copy_(logits)
    out = nss.mb_router(box.t, k)
    torch.cuda.synchronize()
    box.check("logits")
    # NaN above everything, then by falling logit, the lowest index first among equals; -inf is not chosen
    l = box.t.double()
    rank = torch.where(l.isnan(), INF, l)
    top, index = torch.sort(rank, dim=1, descending=True, stable=True)
    index = torch.where(top[:, :k] > -INF, index[:, :k], -1)
    assert torch.equal(out.index.long(), index)
    assert torch.equal(out.counts.long(), torch.bincount(index[index >= 0], minlength=experts))
    assert out.used.item() == int((kind != 5).sum())
    bad = l.isnan().any(1)
    chosen = index >= 0
    assert torch.isnan(out.gate[bad[:, None] & chosen]).all() and not out.gate[~chosen].any() and torch.isnan(out.loss).all()
    assert torch.isfinite(out.gate[~bad]).all()
    clean = (kind == 0) | (kind == 4) | (kind == 5)
    alone = check_router(nss, box.t[clean].contiguous(), k)
    assert torch.equal(out.gate[clean], alone.gate)
