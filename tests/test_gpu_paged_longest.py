"""The paged forward at the longest history that the interface admits (2^31 - 29 tokens), whose last key tile ends at
2^31: the history is one shared page over and over, the last pages are the request's own and NaN past its end.

The count correction (lambda = 1.5, e^32 at this length) leaves the shared keys 2e-5 of a row's weight, so fp32 sums
over 2^31 keys, which may be off by 1e-2 (2^17 additions of one value to a running sum), move no entry by more than
2e-7 max|V|, and the operator's tolerances stand: 1e-5 max|V| (fp32), 1e-2 max|V| (bf16).
"""
import math

import numpy as np
import pytest
import torch

from relation_token_mixing_gb300 import binding as rb

pytestmark = pytest.mark.gpu

PAGE, WIDTH = 16, (1 << 27) - 1
LENGTH = (WIDTH - 1) * PAGE + 3
OWN = 3  # pages at the end


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("fresh", [1, 20])
def test_the_last_tile_of_the_longest_history(fresh, dtype):
    d, lam, tau = 64, 1.5, 1.0
    g = torch.Generator().manual_seed(fresh)
    pools = [torch.randn(1 + OWN, 1, PAGE, d, generator=g).to(dtype) for _ in range(2)]
    for p in pools:
        p[OWN, 0, LENGTH % PAGE:] = float("nan")
    P1 = torch.randn(fresh, 1, d, generator=g).to(dtype)
    table = torch.zeros(1, WIDTH, dtype=torch.int32, device="cuda")
    table[0, -OWN:] = torch.arange(1, 1 + OWN)
    ints = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    Y, _ = rb.paged_fwd(P1.cuda(), *(p.cuda() for p in pools), table, ints(0, fresh), ints(LENGTH - fresh), fresh, tau,
                        lam)
    torch.cuda.synchronize()
    assert rb.relation_check_device_status() == 0
    K, V = (p.double().numpy()[:, 0].reshape(-1, d) for p in pools)
    first = (WIDTH - OWN) * PAGE  # position of the first own page
    pos = np.concatenate([np.zeros(PAGE, dtype=np.int64), first + np.arange(OWN * PAGE)])
    for t in range(fresh):
        i = LENGTH - fresh + t
        U = K @ P1[t, 0].double().numpy() / math.sqrt(d)
        R = U / (1.0 + np.exp(-U)) - lam * math.log(i + 1) + np.where(np.arange(len(pos)) < PAGE, math.log(WIDTH - OWN), 0.0)
        R = np.where(pos == i, 1.0 / (1.0 + np.exp(-U / tau)), R)
        seen = pos <= i
        w = np.exp(R[seen] - R[seen].max())
        want = w @ V[seen] / w.sum()
        err = np.abs(Y[t, 0].double().cpu().numpy() - want).max()
        assert err <= (1e-5 if dtype is torch.float32 else 1e-2) * np.nanmax(np.abs(V)), (t, err)
