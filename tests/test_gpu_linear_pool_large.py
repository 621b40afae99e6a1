"""Chunks whose factors times their states pass float32 although nothing of the result does."""
import numpy as np
import pytest

from linear_pool_cases import check, inputs, on_gpu, packed
from relation_token_mixing_gb300 import binding as rb

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lengths", [[64], [200, 40], [900, 20, 64]])
@pytest.mark.parametrize("d", [64, 60])
@pytest.mark.parametrize("exponent", [20, 40, 90])
def test_large_states_in_fading_chunks(exponent, d, lengths):
    """I~ around 2^exponent where some channels lose 2^190 in a chunk of 64 tokens: the key's factor is up to 2^95."""
    x = inputs(lengths, 2, d, seed=exponent)
    x["G"][:, :, ::3] = -190 / 64 * np.log(2.0)
    x["I"] *= 2.0 ** exponent
    x["states"] *= 2.0 ** exponent
    c = on_gpu(x)
    Y = packed(c, max_fresh=max(lengths))
    assert rb.relation_check_device_status() == 0
    check(x, Y, c["states"])
