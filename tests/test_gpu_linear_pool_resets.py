"""States of strongly fading chunks: tokens that forget everything, side by side, near a warp's and a chunk's end."""
import numpy as np
import pytest

from linear_pool_cases import check, inputs, on_gpu, packed, reference
from relation_token_mixing_gb300 import binding as rb

pytestmark = pytest.mark.gpu

RESETS = {"one": [56], "four": range(56, 60), "six": range(56, 62), "two_warps": range(40, 60), "most": range(2, 61),
          "all_but_the_last": range(0, 63), "the_last": [63], "every_other": range(1, 64, 2), "next_chunk": range(70, 77)}


@pytest.mark.parametrize("gate", [False, True])
@pytest.mark.parametrize("d,lengths", [(64, [64]), (60, [90, 64]), (64, [900, 70])])
@pytest.mark.parametrize("which", list(RESETS))
def test_states_after_resets(which, d, lengths, gate):
    """What a token behind the resets leaves keeps its retention to the end as closely as in any other chunk.

    The state within 2^-15 of the sum of magnitudes: k~ in two parts, 2^-17; the log2-retentions from a key to the
    chunk's end, some 6 at most after the resets here, in up to 15 additions of half of 2^-21 each, 2^-18 with ln 2; the
    state's retention from chunk to chunk, two functions of 2^-22 a chunk and the sum's own roundings, below 2^-17 in 15
    chunks; a sigmoid, a norm and seven products, 2^-20.  Where nothing is left of a channel, 2^-20 of the
    largest state."""
    x = inputs(lengths, 2, d, gate, scale=0.1, seed=len(which))
    for at in RESETS[which]:
        for first in x["starts"][:-1].tolist():
            if first + at < x["G"].shape[0]:
                x["G"][first + at] = 1e4 if gate else -1e9
    c = on_gpu(x)
    Y = packed(c, max_fresh=max(lengths))
    got = c["states"].double().cpu().numpy()
    assert rb.relation_check_device_status() == 0
    check(x, Y, c["states"])
    (_, S), (_, Sa) = reference(x)
    tol = 2.0 ** -15 * Sa + 2.0 ** -20 * float(Sa.max())
    assert (np.abs(got - S) <= tol).all(), float((np.abs(got - S) / tol).max())
