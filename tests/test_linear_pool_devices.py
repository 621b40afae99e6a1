"""The wrappers of Linear Relation over a pool of states refuse a tensor of another device, whichever it is (CPU: tensors
that say so)."""
import pytest
import torch

from linear_pool_cases import TAU, inputs, packed
from relation_token_mixing_gb300 import binding as rb


class Elsewhere(torch.Tensor):
    """A host tensor of the second GPU, as far as a caller can ask."""

    def get_device(self):
        return 1


@pytest.mark.parametrize("which", ["P2", "I", "G", "A_log", "dt_bias", "starts", "states", "slots_in", "slots_out", "Y",
                                   "workspace"])
def test_packed(which):
    x = inputs([2, 1], 2, 64, gate=True)
    more = dict(Y=torch.empty_like(x["P1"]), workspace=torch.empty(1 << 10, dtype=torch.uint8))
    of = more if which in more else x
    of[which] = of[which].as_subclass(Elsewhere)
    with pytest.raises(ValueError, match="one device"):
        packed(x, max_fresh=2, **more)


@pytest.mark.parametrize("which", ["P2", "G", "states", "slots_out", "Y"])
def test_step(which):
    x = inputs([2, 1], 2, 64, gate=True)
    x["Y"] = torch.empty_like(x["P1"])
    x[which] = x[which].as_subclass(Elsewhere)
    with pytest.raises(ValueError, match="one device"):
        rb.linear_step(x["P1"], x["P2"], x["I"], x["G"], x["states"], x["slots_in"], x["slots_out"], TAU, x["A_log"],
                       x["dt_bias"], x["Y"])
