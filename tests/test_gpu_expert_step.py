"""Routing, the experts' products and both steps together, as a training step calls them."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

TOKENS, WIDTH, HIDDEN, EXPERTS, TOP_K = 700, 128, 200, 6, 2


@pytest.fixture(scope="module")
def nss():
    from newton_schulz_stacked_gb300.build import build_all
    build_all()
    import newton_schulz_stacked_gb300 as nss
    return nss


def _inputs(seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    x = torch.randn(TOKENS, WIDTH, generator=g, device="cuda").bfloat16()
    up = (torch.randn(EXPERTS, HIDDEN, WIDTH, generator=g, device="cuda") * WIDTH ** -0.5).bfloat16().requires_grad_()
    down = (torch.randn(EXPERTS, WIDTH, HIDDEN, generator=g, device="cuda") * HIDDEN ** -0.5).bfloat16().requires_grad_()
    bias = (0.1 * torch.randn(EXPERTS, HIDDEN, generator=g, device="cuda")).requires_grad_()
    logits = torch.randn(TOKENS, EXPERTS, generator=g, device="cuda")
    logits[:, 3] = -math.inf                     # an expert that nobody takes
    valid = torch.rand(TOKENS, generator=g, device="cuda") < 0.95
    weight = torch.randn(TOKENS, WIDTH, generator=g, device="cuda")
    return x, up, down, bias, logits, valid, weight


def _forward(linear, x, up, down, bias, routing):
    expert = routing.index.flatten()
    place = expert.masked_fill(expert < 0, EXPERTS).argsort(stable=True)
    token, ends = place // TOP_K, routing.counts.cumsum(0, dtype=torch.int32)
    y = linear(linear(x[token], up, bias, "relu2", ends), down, None, "none", ends)
    return y, token, place


def test_gradients_of_routed_experts(nss):
    from newton_schulz_stacked_gb300 import autograd as A
    x, up, down, bias, logits, valid, weight = _inputs()
    routing = A.route(logits, TOP_K, valid, normalize=True)
    assert routing.counts[3] == 0
    y, token, place = _forward(lambda r, w, b, act, ends: A.linear(r, w, b, activation=act, ends=ends), x, up, down, bias, routing)
    used = int(routing.counts.sum())
    assert used == TOP_K * int(valid.sum()) and not y[used:].any()
    (y.float() * routing.gate.flatten()[place, None] * weight[token]).sum().backward()

    wide = [p.detach().double().requires_grad_() for p in (up, down, bias)]
    loss = 0
    for t in range(TOP_K):
        for e in range(EXPERTS):
            rows = torch.nonzero(routing.index[:, t] == e)[:, 0]
            h = (x[rows].double() @ wide[0][e].T + wide[2][e]).clamp(min=0) ** 2
            loss = loss + ((h @ wide[1][e].T) * routing.gate[rows, t, None].double() * weight[rows].double()).sum()
    loss.backward()
    # roundings of half a step, 2^-8: h (whose slope passes twice its relative error on), dy, dz, the result
    for p, q in zip((up, down, bias), wide):
        assert (p.grad.double() - q.grad).norm() <= 6 * 2.0 ** -8 * q.grad.norm()
        assert not p.grad[3].any()


def test_a_step_of_banks_and_the_rest(nss):
    """The gradients go to the Muon step and to AdamW as they are; a captured step replays with the same bits as eager ones."""
    from newton_schulz_stacked_gb300 import autograd as A

    def fresh():
        x, up, down, bias, logits, valid, weight = _inputs(1)
        banks = [nss.BankState(p.detach(), torch.zeros_like(p), torch.zeros(p.shape, device="cuda"),
                               torch.zeros(p.shape, device="cuda", dtype=torch.int16)) for p in (up, down)]
        adam = nss.adamw_state(bias, torch.zeros_like(bias), bits=8)
        return x, up, down, bias, logits, valid, weight, banks, adam

    def gradients(x, up, down, bias, logits, valid, weight, banks, adam):
        routing = A.route(logits, TOP_K, valid, normalize=True)
        y, token, place = _forward(lambda r, w, b, act, ends: A.linear(r, w, b, activation=act, ends=ends), x, up, down, bias,
                                   routing)
        loss = (y.float() * routing.gate.flatten()[place, None] * weight[token]).sum()
        for g, to in zip(torch.autograd.grad(loss, (up, down, bias)), (banks[0].grad, banks[1].grad, adam.grad)):
            to.copy_(g)

    def step(state, scalars, workspace, adam_workspace, muon):
        gradients(*state)
        with torch.no_grad():
            workspace = nss.muon_multi_step_dev(state[7], muon, workspace=workspace)
            adam_workspace = nss.adamw_multi_step_dev([state[8]], scalars, seed=3, workspace=adam_workspace)
        return workspace, adam_workspace

    muon = torch.tensor([0.02, 0.01, 0.9, 0.95] * 2, device="cuda")
    scalars = torch.tensor([1e-2, 0.0, 0.9, 0.95, 1e-8, 1], dtype=torch.float64, device="cuda")
    eager, graphed = fresh(), fresh()
    workspaces = step(fresh(), scalars, None, None, muon)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(graphed, scalars, *workspaces, muon)
    for i in range(1, 4):
        scalars[5] = i
        graph.replay()
        step(eager, scalars, None, None, muon)
    torch.cuda.synchronize()
    assert nss.mb_sync_status() == 0
    assert not torch.equal(eager[1], _inputs(1)[1])
    for a, b in zip((*(t for k in eager[7] for t in (k.bank, k.momentum, k.mantissa)), eager[3], *eager[8][2:4]),
                    (*(t for k in graphed[7] for t in (k.bank, k.momentum, k.mantissa)), graphed[3], *graphed[8][2:4])):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
