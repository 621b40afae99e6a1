"""What the paged wrappers refuse or arrange before the library is called (CPU)."""
import pytest
import torch

from relation_token_mixing_gb300 import binding as rb


def _i32(*s):
    return torch.zeros(*s, dtype=torch.int32)


def _bf(*s):
    return torch.zeros(*s, dtype=torch.bfloat16)


@pytest.mark.parametrize("theta", [torch.zeros(2, dtype=torch.float64), torch.zeros(2, dtype=torch.bfloat16),
                                   torch.zeros(1), torch.zeros(3), torch.zeros(0)])
def test_store_refuses_a_theta_that_is_not_float32_of_half_the_cache_heads(theta):
    with pytest.raises(ValueError, match="theta"):
        rb.paged_store(_bf(3, 8, 64), _bf(3, 4, 64), _bf(3, 4, 64), theta, 0, 1e4, _i32(3), _i32(3).long(),
                       _bf(3, 8, 64), _bf(8, 4, 16, 64), _bf(8, 4, 16, 64))
