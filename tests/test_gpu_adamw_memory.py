"""Memory that two places of an AdamW call share: refused where it is written, before anything is stepped."""
import pytest
import torch

from test_gpu_adamw import LR, WD, _check, _expect, _state, nss  # noqa: F401

pytestmark = pytest.mark.gpu


def _bytes(states):
    return [t.clone().view(torch.uint8) for s in states for t in s[:7] if t is not None]


@pytest.mark.parametrize("bits", [32, 8])
def test_two_tensors_may_not_share_what_is_written(nss, bits):
    """Any written field of one tensor with any written field, or the gradient, of another."""
    a, b = (_state(nss, 1000, "bf16", "bf16", True, bits, seed=s) for s in (0, 50))
    before = _bytes([a, b])
    shared = [{"param": a.param}, {"exp_avg": a.exp_avg}, {"exp_avg_sq": a.exp_avg_sq}, {"exp_avg": a.exp_avg_sq},
              {"mantissa": a.mantissa}, {"grad": a.param}, {"mantissa": a.param.view(torch.int16)}, {"param": a.grad}]
    if bits == 8:
        shared += [{"avg_scale": a.avg_scale}, {"sq_scale": a.sq_scale}, {"avg_scale": a.sq_scale}]
    else:
        shared += [{"grad": a.exp_avg}]
    for change in shared:
        for pair in ([a, b._replace(**change)], [b._replace(**change), a]):
            with pytest.raises(ValueError, match="overlap"):
                nss.adamw_multi_step(pair, LR, WD)
    # a part of another's memory, among many that are apart
    many = [_state(nss, 64 + i, bits=bits, seed=i) for i in range(60)]
    part = many[40].exp_avg[3:43] if bits == 32 else many[40].exp_avg[1:41]
    small = _state(nss, 40, bits=bits, seed=99)
    with pytest.raises(ValueError, match="exp_avg of tensor 4[01]"):
        nss.adamw_multi_step(many[:20] + [small._replace(exp_avg=part)] + many[20:], LR, WD)
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(before, _bytes([a, b])))


def test_what_is_read_or_written_beside_the_list(nss):
    s = _state(nss, 1000)
    scalars = torch.tensor([LR, WD, 0.9, 0.95, 1e-8, 1], dtype=torch.float64, device="cuda")
    with pytest.raises(ValueError, match="overlap"):
        nss.adamw_multi_step([s], LR, WD, grad_scale=s.exp_avg[5:6])
    with pytest.raises(ValueError, match="overlap"):
        nss.adamw_multi_step_dev([s], scalars, workspace=s.exp_avg_sq.view(torch.uint8))
    held = torch.zeros(64, dtype=torch.float64, device="cuda")           # (a workspace for one tensor is 40 bytes)
    held[4:10] = scalars
    with pytest.raises(ValueError, match="overlap"):
        nss.adamw_multi_step_dev([s], held[4:10], workspace=held.view(torch.uint8))
    with pytest.raises(ValueError, match="overlap"):
        nss.adamw_multi_step_dev([s._replace(grad=s.param)], scalars)
    nss.adamw_multi_step_dev([s], held[4:10], grad_scale=held[20:21].view(torch.float32)[:1], workspace=held[32:].view(torch.uint8))
    assert nss.mb_sync_status() == 0


def test_memory_side_by_side_and_shared_gradients(nss):
    """Views of flat buffers in any order, and tensors that share one gradient, are stepped as ever."""
    flat = [_state(nss, 6000, seed=7), _state(nss, 6000, seed=7)]
    cuts = [(4000, 6000), (0, 1), (1, 1500), (1500, 4000)]
    pieces = [nss.AdamState(*(t[a:b] for t in flat[0][:4])) for a, b in cuts]
    want = [_expect(p, i, 3) for i, p in enumerate(pieces)]
    nss.adamw_multi_step(pieces, LR, WD, 0.9, 0.95, 1e-8, 3)
    for p, w in zip(pieces, want):
        _check(p, w)
    states = [_state(nss, 512, seed=s) for s in (0, 10)]
    states = [s._replace(grad=states[0].grad) for s in states]
    want = [_expect(s, i, 2) for i, s in enumerate(states)]
    nss.adamw_multi_step(states, LR, WD, 0.9, 0.95, 1e-8, 2)
    for s, w in zip(states, want):
        _check(s, w)


def test_memory_in_any_order(nss):
    """Fields that ascend, descend or do neither over the list, one within another's gaps, a factor between them: stepped where all
    are apart, refused where two share a byte."""
    whole = torch.zeros(4 * 64 * 24, device="cuda")
    cells = whole.view(24, 4, 64)                # cell i: a param, a grad and two moments side by side
    orders = [list(range(20)), list(range(19, -1, -1)), [7, 3, 11, 0, 19, 5, 2, 13, 1, 17, 4, 16, 6, 10, 8, 18, 9, 12, 14, 15]]
    factor = cells[22, 1, 10:11]
    for a in orders:
        for b in orders:
            whole.normal_().abs_()
            factor.fill_(0.5)
            states = [nss.AdamState(cells[i, 0], cells[j, 1], cells[j, 2], cells[i, 3]) for i, j in zip(a, b)]
            want = [_expect(s, p, 2, 0.5) for p, s in enumerate(states)]
            nss.adamw_multi_step(states, LR, WD, 0.9, 0.95, 1e-8, 2, grad_scale=factor)
            for s, w in zip(states, want):
                _check(s, w)
            for bad in (states[11]._replace(exp_avg=whole.view(-1)[whole.view(-1).shape[0] - 64:]),
                        states[11]._replace(exp_avg=cells[a[3], 3].flatten()), states[11]._replace(param=cells[b[2], 1]),
                        states[11]._replace(grad=cells[21, 2])):
                listed = states[:11] + [bad] + states[12:]
                shares = bad.exp_avg.data_ptr() == states[3].exp_avg_sq.data_ptr() or bad.param.data_ptr() == states[2].grad.data_ptr()
                if shares:
                    with pytest.raises(ValueError, match="overlap"):
                        nss.adamw_multi_step(listed, LR, WD, grad_scale=factor)
                else:
                    nss.adamw_multi_step(listed, LR, WD, grad_scale=factor)
            with pytest.raises(ValueError, match="grad_scale"):
                nss.adamw_multi_step(states, LR, WD, grad_scale=states[5].exp_avg[63:])


def test_a_scalar_clipping_factor(nss):
    """What a norm gives has no dimension: the same step as from one value in a row, by value and from the device."""
    states = [_state(nss, 3000, bits=b) for b in (32, 32, 32)]
    factor = torch.full((2, 2), 0.25, device="cuda").norm()               # 0.5
    assert factor.dim() == 0
    scalars = torch.tensor([LR, WD, 0.9, 0.95, 1e-8, 4], dtype=torch.float64, device="cuda")
    want = _expect(states[0], 0, 4, 0.5)
    nss.adamw_multi_step([states[0]], LR, WD, 0.9, 0.95, 1e-8, 4, grad_scale=factor)
    nss.adamw_multi_step([states[1]], LR, WD, 0.9, 0.95, 1e-8, 4, grad_scale=factor.reshape(1))
    nss.adamw_multi_step_dev([states[2]], scalars, grad_scale=factor)
    for s in states:
        _check(s, want)
    for bad in (torch.ones(2, device="cuda"), torch.ones(1, 1, device="cuda"), torch.ones((), device="cuda", dtype=torch.float64),
                torch.ones(())):
        with pytest.raises(ValueError, match="grad_scale"):
            nss.adamw_multi_step(states, LR, WD, grad_scale=bad)
