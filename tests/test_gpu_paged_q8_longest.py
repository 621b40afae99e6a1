"""The forward over 8-bit pages at the longest history that the interface admits, as for bf16 pages: one shared page over
and over, the last pages the request's own, with NaN scales past its end.

The count correction (lambda = 1.5, e^32 at this length) leaves the shared keys 2e-5 of a row's weight, so sums over 2^31
keys in fp32 move no entry by more than 2e-7 max|I~|, and the operator's 1e-2 max|I~| stands (against the rows as kept)."""
import math

import numpy as np
import pytest
import torch

from paged_q8_cases import quantised
from relation_token_mixing_gb300 import binding as rb
from test_gpu_paged_longest import LENGTH, OWN, PAGE, WIDTH

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fresh", [1, 20])
def test_the_last_tile_of_the_longest_history(fresh):
    d, lam, tau = 64, 1.5, 1.0
    g = torch.Generator().manual_seed(fresh)
    pools = [torch.randn(1 + OWN, 1, PAGE, d, generator=g).bfloat16() for _ in range(2)]
    for p in pools:
        p[OWN, 0, LENGTH % PAGE:] = float("nan")
    (k, ks, K), (v, vs, V) = (quantised(p, d, g) for p in pools)
    P1 = torch.randn(fresh, 1, d, generator=g).bfloat16()
    table = torch.zeros(1, WIDTH, dtype=torch.int32, device="cuda")
    table[0, -OWN:] = torch.arange(1, 1 + OWN)
    ints = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    Y, _ = rb.paged_fwd_q8(P1.cuda(), k.cuda(), v.cuda(), torch.stack([ks, vs], -1).cuda(), table, ints(0, fresh),
                           ints(LENGTH - fresh), fresh, tau, lam)
    torch.cuda.synchronize()
    assert rb.relation_check_device_status() == 0
    K, V = (x.numpy()[:, 0].reshape(-1, d) for x in (K, V))
    first = (WIDTH - OWN) * PAGE  # position of the first own page
    pos = np.concatenate([np.zeros(PAGE, dtype=np.int64), first + np.arange(OWN * PAGE)])
    for t in range(fresh):
        i = LENGTH - fresh + t
        seen = pos <= i
        U = K[seen] @ P1[t, 0].double().numpy() / math.sqrt(d)
        R = U / (1.0 + np.exp(-U)) - lam * math.log(i + 1)
        R += np.where(np.arange(len(U)) < PAGE, math.log(WIDTH - OWN), 0.0)
        R = np.where(pos[seen] == i, 1.0 / (1.0 + np.exp(-U / tau)), R)
        w = np.exp(R - R.max())
        want = w @ V[seen] / w.sum()
        err = np.abs(Y[t, 0].double().cpu().numpy() - want).max()
        assert err <= 1e-2 * np.nanmax(np.abs(V)), (t, err)
