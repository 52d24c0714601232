"""Refusals of the block operators under autograd that need no device."""
import pytest
import torch


@pytest.mark.parametrize("which", ["positions", "inv_freq"])
def test_rotary_refuses_to_lose_a_gradient(which):
    """The angles' factors have no gradient; one that is to be trained is refused, not left untrained."""
    from newton_schulz_stacked_gb300 import autograd as A
    at = {"positions": torch.zeros(1, 1, 3), "inv_freq": torch.ones(4)}
    at[which].requires_grad_()
    q = torch.zeros(1, 3, 2, 8)
    with pytest.raises(ValueError, match=f"{which} requires a gradient"):
        A.rotary(q, None, at["positions"], at["inv_freq"], (4,))
    with torch.no_grad(), pytest.raises(ValueError, match="must be a CUDA tensor"):     # goes on to the call itself
        A.rotary(q, None, at["positions"], at["inv_freq"], (4,))
    with pytest.raises(ValueError, match="must be a CUDA tensor"):
        A.rotary(q, None, at["positions"].detach(), at["inv_freq"].detach(), (4,))
