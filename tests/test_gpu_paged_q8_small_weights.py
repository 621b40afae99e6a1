"""The forward over 8-bit pages with few rows: weights far below the largest, so many that they matter together."""
import math

import pytest
import torch

from relation_token_mixing_gb300 import binding as rb

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("U", [16.75, 17.5])
@pytest.mark.parametrize("d", [64, 128])
def test_a_million_small_weights_under_a_large_one(d, U):
    """One key of score U, whose state is 0, and 2^20 - 1 of score 0, whose states are 1; as many requests over the same
    pages as the kernel has workers, so that each worker has a whole history and one reference.

    The small weights are 2^-24.2 and 2^-25.2 of the large one: under float16's least step, 2^-24, if the reference were
    float16's 1.  Y = n e^-U / (1 + n e^-U).  Its error: 2^-8 of itself for the output and 2^-11 for the weights, the
    exponential's (U/2) 2^-10.9, and half of float16's least step under a reference at 2^7, 2^-32, for each of n."""
    page, pages, H = 256, 4096, 1
    n = page * pages - 1  # cached; the request's new token is the last
    workers = 12 * torch.cuda.get_device_properties(0).multi_processor_count
    P2, I, scales = rb.paged_pages_q8(pages, 1, page, d)
    I.fill_(64)
    scales[..., 1] = 2.0 ** -6
    scales[..., 0] = 1.0
    I[0, 0, 0] = 0
    P2[0, 0, 0, 0] = 67 if U == 16.75 else 70  # P1's first column makes it U
    P1 = torch.zeros(workers, H, d, dtype=torch.bfloat16, device="cuda")
    P1[..., 0] = 2.0 if d == 64 else 2.0 * math.sqrt(2.0)
    u = float(P1[0, 0, 0]) * float(P2[0, 0, 0, 0]) / math.sqrt(d)
    table = torch.arange(pages, dtype=torch.int32, device="cuda").repeat(workers, 1)
    starts = torch.arange(workers + 1, dtype=torch.int32, device="cuda")
    cached = torch.full((workers,), n, dtype=torch.int32, device="cuda")
    Y, _ = rb.paged_fwd_q8(P1, P2, I, scales, table, starts, cached, 1, 1.0, 0.0)
    torch.cuda.synchronize()
    assert rb.relation_check_device_status() == 0
    R = u / (1 + math.exp(-u))
    small = (n - 1 + math.exp(0.5)) * math.exp(-R)
    want = small / (1 + small)
    tol = want * (2.0 ** -8 + 2.0 ** -11 + u / 2 * 2.0 ** -10.9) + n * 2.0 ** -32
    assert tol < 0.1 * want
    off = (Y.double() - want).abs().max()
    assert float(off) <= tol, (float(off), tol, want)
