"""What one token leaves in a state: the key in three bf16 parts, which two parts would not give."""
import numpy as np
import pytest
import torch

from linear_pool_cases import inputs, on_gpu, packed, reference
from relation_token_mixing_gb300 import binding as rb

pytestmark = pytest.mark.gpu

# In units of 2^-24 of the value: the sigmoid 4 (an exponential, a sum, a quotient), 1 / |p2| 6 (four steps of a sum and a
# square root), the key's factor and the state's two functions of 3 each and 1 for the exponents, six products 6, the
# three parts 1 and their sum in the accumulator 6: 30, below 2^-19.
BOUND = 2.0 ** -19


def _bf16(x):
    return torch.from_numpy(x).float().bfloat16().double().numpy()


@pytest.mark.parametrize("d,lengths", [(64, [40, 64]), (60, [17, 50, 64]), (48, [100, 33]), (64, [900, 64])])
def test_a_state_of_one_token(d, lengths):
    """I~ is zero but for each request's last token but one, so the state is one product and no error averages out."""
    H = 4
    x = inputs(lengths, H, d, scale=0.02, slots=([-1] * len(lengths), list(range(len(lengths)))), seed=d)
    keep = torch.zeros(x["I"].shape[0], 1, 1)
    keep[(x["starts"][1:] - 2).tolist()] = 1
    x["I"] = x["I"] * keep.bfloat16()
    c = on_gpu(x)
    packed(c, max_fresh=max(lengths))
    got = c["states"].double().cpu().numpy()
    assert rb.relation_check_device_status() == 0
    (_, S), _ = reference(x)
    used = S[: len(lengths)]
    off = np.abs(got[: len(lengths)] - used)
    assert (off <= BOUND * np.abs(used)).all(), float((off / np.maximum(np.abs(used), 1e-30)).max() / BOUND)
    # The test would notice: these states with their keys in two parts are off by more.
    q = used[0] / np.abs(used[0]).max()
    two = _bf16(q) + _bf16(q - _bf16(q))
    assert (np.abs(two - q) > BOUND * np.abs(q)).any()
