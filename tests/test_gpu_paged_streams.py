"""The paged forward on a stream of its own while the caller's stream goes on allocating."""
import pytest
import torch

from relation_token_mixing_gb300 import binding as rb
from test_gpu_paged import FWD, Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("name", ["decode_long", "mixed", "f32_d64"])
def test_own_allocations_outlive_the_kernels(name):
    """The side stream has work queued before the forward; meanwhile the caller's stream takes and fills tensors of
    the sizes that the call allocated and freed."""
    case = Case(**FWD[name])
    dev = [x.cuda() for x in (case.P1, *case.pools, case.table, case.starts, case.cached)]
    most = max(f for _, f in case.rows)
    prob = rb.paged_for(dev[0], dev[1], len(case.rows), case.table.shape[1], case.tau, case.lam, case.layout)
    size = rb.relation_paged_workspace_bytes(prob, most)
    want, _ = rb.paged_fwd(*dev, most, case.tau, case.lam, layout=case.layout)
    want = want.clone()
    side, a = torch.cuda.Stream(), torch.randn(4096, 4096, device="cuda")
    for _ in range(3):
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            for _ in range(20):
                b = a @ a
        Y, _ = rb.paged_fwd(*dev, most, case.tau, case.lam, layout=case.layout, stream=side)
        others = [torch.full((size // 4,), float("nan"), device="cuda") for _ in range(4)]
        others += [torch.full_like(dev[0], float("nan")) for _ in range(4)]
        torch.cuda.synchronize()
        assert rb.relation_check_device_status() == 0
        n = int(case.starts[-1])
        assert torch.equal(Y[:n], want[:n])
    del others, b
