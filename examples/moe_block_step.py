"""Trains one mixture-of-experts block over image patches with the Muon step.

The block's matrices live in stacked banks (q/k/v/o, the experts' two products, the router's
gate), which muon_multi_step updates in place; what stands between the products is this
library's: layer norm, rotary positions over (height, width), expert routing with its balance
loss, each through its gradient.  The products and the attention are torch's.

    python examples/moe_block_step.py [--steps 30]

Prints the task's loss, the balance loss and the experts' counts, and fails unless the task's
loss falls.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import newton_schulz_stacked_gb300 as nss                          # noqa: E402
from newton_schulz_stacked_gb300 import autograd as block          # noqa: E402

BATCH, GRID, WIDTH, HEADS, DIM, EXPERTS, TOP_K, HIDDEN = 8, 14, 256, 4, 64, 8, 2, 512
TOKENS = GRID * GRID


def bank(shape, gen):
    """A bank's state: bf16 weights (the high halves of fp32 ones), their low halves, momentum."""
    w = torch.randn(shape, generator=gen, device="cuda") * shape[-1] ** -0.5
    halves = w.view(torch.int16)                                   # low, high, low, high, ...
    weight = halves[..., 1::2].contiguous().view(torch.bfloat16).requires_grad_()
    mantissa = halves[..., 0::2].contiguous()
    return {"weight": weight, "mantissa": mantissa, "momentum": torch.zeros(shape, device="cuda")}


def forward(x, banks, norms, positions, inv_freq):
    q_w, k_w, v_w, o_w = banks["attn"]["weight"]
    h = block.layer_norm(x, *norms[0])
    q, k, v = ((h @ w.T).view(BATCH, TOKENS, HEADS, DIM) for w in (q_w, k_w, v_w))
    q, k = block.rotary(q, k, positions, inv_freq, (DIM // 4, DIM // 4))
    scores = torch.einsum("bqhd,bkhd->bhqk", q, k).float() * DIM ** -0.5
    mix = torch.einsum("bhqk,bkhd->bqhd", scores.softmax(-1).to(x.dtype), v)
    x = x + mix.reshape(BATCH, TOKENS, WIDTH) @ o_w.T

    h = block.layer_norm(x, *norms[1]).view(-1, WIDTH)
    routing = block.route(h @ banks["gate"]["weight"][0].T, TOP_K, normalize=True)
    out = torch.zeros_like(h, dtype=torch.float32)
    for e in range(EXPERTS):
        token, place = torch.nonzero(routing.index == e, as_tuple=True)
        y = torch.relu(h[token] @ banks["up"]["weight"][e].T).square() @ banks["down"]["weight"][e].T
        out = out.index_add(0, token, y.float() * routing.gate[token, place, None])
    return x + out.view_as(x).to(x.dtype), routing


def train(steps=30, lr=0.02, balance=0.01, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    banks = {"attn": bank((4, WIDTH, WIDTH), gen), "up": bank((EXPERTS, HIDDEN, WIDTH), gen),
             "down": bank((EXPERTS, WIDTH, HIDDEN), gen), "gate": bank((1, EXPERTS, WIDTH), gen)}
    norms = [(torch.ones(WIDTH, device="cuda", requires_grad=True), torch.zeros(WIDTH, device="cuda", requires_grad=True))
             for _ in range(2)]
    at = torch.arange(TOKENS, device="cuda")
    positions = torch.stack((at // GRID, at % GRID)).to(torch.int32)
    inv_freq = (100.0 ** (-torch.arange(DIM // 4, device="cuda") / (DIM // 4))).repeat(2)
    # the task: every patch answers with a fixed linear map of its upper neighbour
    x = torch.randn((BATCH, TOKENS, WIDTH), generator=gen, device="cuda").bfloat16()
    mix = torch.randn((WIDTH, WIDTH), generator=gen, device="cuda") * WIDTH ** -0.5
    goal = x.float().view(BATCH, GRID, GRID, WIDTH).roll(1, dims=1).reshape(x.shape) @ mix
    workspace, losses = None, []
    for step in range(steps):
        y, routing = forward(x, banks, norms, positions, inv_freq)
        task = (y.float() - goal).square().mean()
        (task + balance * routing.loss).backward()
        with torch.no_grad():
            states = [nss.BankState(b["weight"].detach(), b["weight"].grad, b["momentum"], b["mantissa"])
                      for b in banks.values()]
            workspace = nss.muon_multi_step(states, lr, 0.01, 0.9, workspace=workspace)
            for p in (p for norm in norms for p in norm):
                p -= 0.1 * p.grad
                p.grad = None
            for b in banks.values():
                b["weight"].grad = None
        losses.append((task.item(), routing.loss.item()))
        if step % 5 == 0 or step == steps - 1:
            print(f"step {step:3d}  task {losses[-1][0]:.4f}  balance {losses[-1][1]:.4f}  counts {routing.counts.tolist()}")
    if nss.mb_sync_status() != 0:
        raise RuntimeError("device-side status set after the steps")
    return losses


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=30)
    got = train(ap.parse_args().steps)
    sys.exit(0 if got[-1][0] < 0.9 * got[0][0] else "the task's loss did not fall")
