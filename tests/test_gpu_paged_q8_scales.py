"""The forward over 8-bit pages with the largest and the least scales side by side."""
import numpy as np
import pytest
import torch

from paged_q8_cases import Q8Case
from relation_token_mixing_gb300 import binding as rb

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("rows", [[(64, 2)], [(64, 40)]])
def test_a_row_of_the_least_scale_beside_one_of_a_huge_scale(rows, d):
    """Key 5 has a scale of 2^115 and key 6 one of 2^-126: each is what its own numbers say."""
    case = Q8Case(rows=rows, H=1, G=1, d=d)
    k, v, s = case.q8
    page = int(case.table[0, 0])
    k[:, :, :, :2] = 0
    s[page, 0, 5, 0], s[page, 0, 6, 0] = 2.0 ** 115, 2.0 ** -126
    k[page, 0, 5], k[page, 0, 6] = 0, 0
    k[page, 0, 5, 1], k[page, 0, 6, 0] = 127, 100
    case.P1 = torch.zeros_like(case.P1)  # the queries see column 0 only, which key 6 alone has
    case.P1[..., 0] = 2.0 ** 123
    live = torch.isfinite(s[..., 0].float())
    case.pools = torch.where(live[..., None], k[..., :d].double() * s[..., :1].double(), float("nan")), case.pools[1]
    Y, L = case.run()
    assert rb.relation_check_device_status() == 0
    U = 100 * 2.0 ** -3 / np.sqrt(d)
    R = U / (1 + np.exp(-U))
    states = np.nan_to_num(case.pools[1].numpy())[case.table[0].long().numpy(), 0].reshape(-1, d)
    for t in range(rows[0][1]):
        i = rows[0][0] + t  # before it: 0 but for key 6's; its own: sigmoid(0), the count correction moved to it
        r = np.zeros(i + 1)
        r[6], r[i] = R, 0.5 + case.lam * np.log(i + 1)
        w = np.exp(r)
        assert abs(float(L[t, 0]) - (np.log(w.sum()) - case.lam * np.log(i + 1))) <= 2e-3  # tanh to 2^-11, of which the
        w /= w.sum()                                                                       # own key has a half
        off = np.abs(Y[t, 0].double().numpy() - w @ states[: i + 1])
        # The output's rounding, the weights' (2^-8 or finer), and a tanh of 2^-10.9 in key 6's and the own score.
        assert (off <= 2.0 ** -8 * np.abs(w @ states[: i + 1]) + (2.0 ** -8 + 2.0 ** -10) * (w @ np.abs(states[: i + 1]))).all()
