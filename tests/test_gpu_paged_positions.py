"""The paged store's RoPE at positions that a float32 does not hold, against the float64 oracle.

Tolerance: that of the stored rows (2e-6 max|x| in fp32, 2^-8 max|x| in bf16) and what the angle may be off by, p 2^-49
for the frequency as two floats and p 2^-52 for the oracle's own, together below p 2^-48, times |(a, b)| <= sqrt(2) max|x|.
"""
import numpy as np
import pytest
import torch

from oracle import paged as po
from relation_token_mixing_gb300 import binding as rb

pytestmark = pytest.mark.gpu

POSITIONS = [0, 1, 40000, (1 << 24) - 1, 1 << 24, (1 << 24) + 1, (1 << 24) + 3, (1 << 25) + 1, (1 << 25) + 2, 123456789,
             (1 << 30) + 1, (1 << 30) + 33, (1 << 31) - 130, (1 << 31) - 1]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("d", [48, 60, 64, 80, 128])
def test_store_at_large_positions(d, dtype):
    g = torch.Generator().manual_seed(d)
    N, H, G, page = len(POSITIONS), 4, 2, 16
    X1, X2, I = (torch.randn(N, h, d, generator=g).to(dtype) for h in (H, G, G))
    pools = rb.paged_pages(2, G, page, d, dtype)
    P1 = torch.empty_like(X1, device="cuda")
    rb.paged_store(X1.cuda(), X2.cuda(), I.cuda(), None, 0, 1e4, torch.tensor(POSITIONS, dtype=torch.int32).cuda(),
                   torch.arange(N).cuda(), P1, *pools)
    torch.cuda.synchronize()
    assert rb.relation_check_device_status() == 0
    zeros = [np.zeros(p.shape) for p in pools]
    ref, ref_pages, _ = po.store(X1.double(), X2.double(), I.double(), None, 0, 1e4, POSITIONS, range(N), *zeros, page,
                                 po.BHTD)
    top1, top2 = (float(x.double().abs().max()) for x in (X1, X2))
    for n, p in enumerate(POSITIONS):
        tol = (2e-6 if dtype is torch.float32 else 2.0 ** -8) + 2 ** 0.5 * p * 2.0 ** -48
        got = po.row_of(pools[0].double().cpu().numpy(), n, slice(None), page, po.BHTD)[:, :d]
        want = po.row_of(ref_pages, n, slice(None), page, po.BHTD)[:, :d]
        assert np.abs(P1[n].double().cpu().numpy() - ref[n]).max() <= tol * top1, p
        assert np.abs(got - want).max() <= tol * top2, p
