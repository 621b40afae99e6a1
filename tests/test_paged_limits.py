"""Limits of the paged forward that are refused on the host (CPU; every call here is refused for one reason or another,
so none reaches a GPU)."""
import pytest

from relation_token_mixing_gb300 import binding as rb
from test_paged_pins import A, _fwd, _prob

MISALIGNED = dict(ws=64 * A + 8)  # refused after the limits: 3


@pytest.mark.parametrize("max_fresh,code", [((1 << 21) - 1, 3), (1 << 21, 2), (1 << 22, 2), (0, 2), ((1 << 31) - 1, 2)])
def test_packed_rows_of_a_request_are_counted_in_32_bits(max_fresh, code):
    """Groups of 1024: 2^21 new tokens are 2^31 packed rows, which no kernel of the forward would take up."""
    p = _prob(H=1024, G=1, N=1 << 22)
    assert _fwd(p, max_fresh=max_fresh, **MISALIGNED) == code
    if code == 2:
        assert rb.relation_paged_workspace_bytes(p, max_fresh) == 0


def test_the_bound_of_a_short_batch_is_its_own():
    assert _fwd(_prob(H=1024, G=1, N=1000), max_fresh=0, **MISALIGNED) == 3
