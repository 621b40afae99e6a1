"""Cut calls of Linear Relation over a pool of states (requests above 640 tokens) with values that cannot be followed:
reported, the others' rows and states right, and nothing written behind the workspace."""
import pytest
import torch

from linear_pool_cases import TAU, check, inputs, on_gpu, packed
from relation_token_mixing_gb300 import binding as rb

pytestmark = pytest.mark.gpu
GUARD = 32 << 20


def _cut(c, max_fresh=0):
    """The call with a workspace of the bytes that it needs, inside a larger one that has to stay as it is."""
    prob = rb.linear_packed_for(c["P1"], c["states"], c["slots_in"].numel(), TAU)
    need = rb.relation_linear_packed_workspace_bytes(prob, max_fresh)
    assert need > 0
    ws = torch.full((need + GUARD,), 0x5A, dtype=torch.uint8, device="cuda")
    Y = torch.full_like(c["P1"], 7.0)
    packed(c, max_fresh=max_fresh, Y=Y, workspace=ws[:need])
    torch.cuda.synchronize()
    assert rb.relation_last_launch_count() == 4
    assert (ws[need:] == 0x5A).all()
    return Y, rb.relation_check_device_status()


@pytest.mark.parametrize("times", [2, 3, 5, 100])
@pytest.mark.parametrize("N,H,d", [(1400, 2, 60), (32768, 2, 48), (9000, 8, 64)])
def test_rows_that_come_again_are_skipped(N, H, d, times):
    """Offsets 0, N, 0, N, ...: the first request runs; the others, all with its rows, leave their states alone."""
    R = 2 * times - 1
    x = inputs([N], H, d, slots=(list(range(R)), list(range(R, 2 * R))), seed=times)
    first = {k: t[:1] if k in ("slots_in", "slots_out") else t for k, t in x.items()}
    c = on_gpu(x)
    c["starts"] = torch.tensor([0, N] * times, dtype=torch.int32, device="cuda")
    Y, status = _cut(c)
    assert status == 1 and rb.relation_check_device_status() == 0
    check(first, Y, c["states"])


@pytest.mark.parametrize("what", ["past", "descending", "bound", "slot_in", "slot_out"])
def test_values_that_cannot_be_followed_are_reported(what):
    x = inputs([900, 3, 1200], 2, 64, slots=([0, 1, 2], [3, 4, 5]), seed=13)
    before = x["states"].clone()
    c = on_gpu(x)
    if what == "past":
        c["starts"][3] = 2104
    elif what == "descending":  # the second request's; the third then has the first's last rows as well
        c["starts"][1], c["starts"][2] = 903, 700
    elif what == "slot_in":
        c["slots_in"][2] = 6
    elif what == "slot_out":
        c["slots_out"][2] = 1 << 30
    Y, status = _cut(c, 1000 if what == "bound" else 0)
    assert status == 1 and rb.relation_check_device_status() == 0
    states = c["states"].cpu()
    if what in ("past", "bound"):  # the third request is skipped, the others are not
        assert (Y[903:] == 7.0).all() and torch.equal(states[5], before[5])
        x["starts"][3] = 903
        x["slots_out"][2] = -1
        check(x, Y, c["states"])
    elif what == "descending":
        assert torch.equal(states[4], before[4]) and torch.equal(states[5], before[5])
        assert (Y[903:] == 7.0).all()
        x["starts"] = torch.tensor([0, 903], dtype=torch.int32)
        x["slots_in"], x["slots_out"] = x["slots_in"][:1], x["slots_out"][:1]
        check(x, Y, c["states"])
    elif what == "slot_in":  # as a new request
        x["slots_in"][2] = -1
        check(x, Y, c["states"])
    else:
        x["slots_out"][2] = -1
        check(x, Y, c["states"])


def test_an_empty_request_between_the_rows_of_others():
    """Offsets that stand still are no descent: nothing is reported, the states of requests without tokens are copied."""
    x = inputs([700, 0, 0, 900, 0, 5], 2, 64, seed=21)
    c = on_gpu(x)
    Y, status = _cut(c)
    assert status == 0
    check(x, Y, c["states"])
