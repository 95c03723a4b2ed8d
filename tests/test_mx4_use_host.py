"""How the 4-bit copies are kept and handed out, without a GPU."""
import pytest
import torch

from elementwise_optimizer_b200 import optim


def test_copies_only_of_the_optimizers_own_parameters():
    """A tensor that no step of this optimizer writes has no copies here,
    whatever its dimensions: they would go stale unnoticed."""
    own, foreign = (torch.nn.Parameter(torch.zeros(4, 4)) for _ in range(2))
    for mx4 in (True, [own]):
        opt = optim.AdamW32bit([own], mx4=mx4)
        with pytest.raises(ValueError, match="not a parameter of this optimizer"):
            opt.mx4_copies(foreign)
        with pytest.raises(ValueError, match="not a parameter of this optimizer"):
            opt.mx4_copies(own.detach())
        assert not opt._mx4_pairs
