"""The forward over 8-bit pages with few rows at scores where one step of float32 is 16 in units of log2: float16 holds
the weights whatever the rounding of their reference."""
import pytest
import torch

from relation_token_mixing_gb300 import binding as rb

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d,scale", [(64, 1.0), (128, 2.0 ** 0.5)])
def test_states_of_a_larger_scale_at_scores_above_2_to_the_27(d, scale):
    """Every key has one score, k 2^20 (2^27 to 2^28 in units of log2) for request k; every other tile has a key whose state
    is 2^16, the others' are 1.  All weights are equal, so Y is the mean: 2^-8 for the output, 2^-11 for the weights."""
    page, pages, ks = 64, 8, list(range(90, 128))
    P2, I, scales = rb.paged_pages_q8(pages, 1, page, d)
    n = page * pages - 1
    P2[..., 0] = 64
    I.fill_(1)
    scales.fill_(1.0)
    big = torch.arange(40, n, 64)
    scales[big // page, 0, big % page, 1] = 2.0 ** 16
    P1 = torch.zeros(len(ks), 1, d, dtype=torch.bfloat16, device="cuda")
    P1[:, 0, 0] = torch.tensor([k * 2.0 ** 17 * scale for k in ks])
    table = torch.arange(pages, dtype=torch.int32, device="cuda").repeat(len(ks), 1)
    starts = torch.arange(len(ks) + 1, dtype=torch.int32, device="cuda")
    cached = torch.full((len(ks),), n, dtype=torch.int32, device="cuda")
    Y, _ = rb.paged_fwd_q8(P1, P2, I, scales, table, starts, cached, 1, 1.0, 0.0)
    torch.cuda.synchronize()
    assert rb.relation_check_device_status() == 0
    want = (n - len(big) + len(big) * 2.0 ** 16) / n
    assert torch.isfinite(Y.float()).all()
    assert float((Y.double() / want - 1).abs().max()) <= 2.0 ** -8 + 2.0 ** -11
