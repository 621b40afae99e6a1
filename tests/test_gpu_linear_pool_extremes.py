"""Linear Relation over a pool of states at the ends of its inputs' ranges: infinities that the formulas take, vectors of
very large and very small norms."""
import numpy as np
import pytest
import torch

from linear_pool_cases import check, inputs, on_gpu, packed, reference
from relation_token_mixing_gb300 import binding as rb

pytestmark = pytest.mark.gpu
LENGTHS = [[12, 3], [90, 20], [900, 40]]


@pytest.mark.parametrize("lengths", LENGTHS)
@pytest.mark.parametrize("gate", [False, True])
@pytest.mark.parametrize("d", [64, 60])
def test_retention_of_nothing_and_of_everything_by_infinities(d, gate, lengths):
    """A log-retention of -infinity forgets a channel; a gate's input of -infinity keeps it, of infinity forgets it."""
    x = inputs(lengths, 2, d, gate, seed=1)
    x["G"][5, 0, ::3] = float("inf") if gate else float("-inf")
    x["G"][7, 1] = float("-inf")
    x["G"][lengths[0] + 1, :, 7] = float("inf") if gate else float("-inf")
    c = on_gpu(x)
    Y = packed(c, max_fresh=max(lengths))
    assert rb.relation_check_device_status() == 0
    assert torch.isfinite(Y.float()).all() and torch.isfinite(c["states"]).all()
    check(x, Y, c["states"])


@pytest.mark.parametrize("lengths", LENGTHS)
def test_an_infinite_query_is_its_token_s_alone(lengths):
    """p1 with an infinity has no direction, so its token's output is NaN; S is 0 or 1, and the state goes on."""
    x = inputs(lengths, 2, 64, seed=2)
    for at, value in ((4, float("inf")), (lengths[0] + 2, float("-inf"))):
        x["P1"][at, 1, 9] = value
    c = on_gpu(x)
    Y = packed(c, max_fresh=max(lengths))
    assert rb.relation_check_device_status() == 0
    (Yr, S), _ = reference(x)
    assert np.isfinite(S).all()
    assert np.array_equal(np.isnan(Y.float().cpu().numpy()), np.isnan(Yr))
    # Without those two tokens' outputs the rest is as ever: their queries as any finite vector that leaves S as it is.
    y = {k: t for k, t in x.items()}
    y["P1"] = x["P1"].clone()
    for at, value in ((4, 1e4), (lengths[0] + 2, -1e4)):
        y["P1"][at, 1] = 0
        y["P1"][at, 1, 9] = value
        assert abs(float(x["P2"][at, 1, 9])) > 1e-2
    (Yy, Sy), _ = reference(y)
    assert np.allclose(Sy, S)
    got = Y.clone()
    for at in (4, lengths[0] + 2):
        got[at, 1] = torch.from_numpy(Yy[at, 1]).bfloat16().cuda()
    check(y, got, c["states"])


@pytest.mark.parametrize("lengths", LENGTHS)
@pytest.mark.parametrize("exponent", [40, 58, -58])
def test_norms_far_from_one(exponent, lengths):
    x = inputs(lengths, 2, 60, seed=3)
    x["P1"] *= 2.0 ** exponent
    x["P2"] *= 2.0 ** -exponent
    c = on_gpu(x)
    Y = packed(c, max_fresh=max(lengths))
    assert rb.relation_check_device_status() == 0
    check(x, Y, c["states"])
