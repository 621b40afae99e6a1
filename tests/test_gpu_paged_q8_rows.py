"""The forward over 8-bit pages held row by row: bounds that follow a row's own sum of weighted states, so that a row
of a long history, whose output is far below the largest state, is checked as closely as any other."""
import math

import numpy as np
import pytest
import torch

from paged_q8_cases import Q8Case
from relation_token_mixing_gb300 import binding as rb
from test_gpu_paged import BHTD, BTHD, FWD, LONG

pytestmark = pytest.mark.gpu


def rows_of(case, only):
    """(packed row, head, Y, the bound of its error) of the packed rows `only`, in 64 bits.

    A weight's relative error: U/2 from products that are exact, summed in float32 in up to 9 steps of 2^-23 of what
    stands there, which with few rows has 1152 |p1| s on it (s: the key's scale, |p1| the sum of absolute values), and
    2^-25 of the row's largest |p1| lost a column; tanh to 2^-10.9 of itself in U/2 (1 + tanh); 6 roundings of the
    exponents, 2^-24 of the larger of |R| and the row's reference each; the weight's own rounding, 2^-11 (float16, or 2^-32
    of the largest product of a weight and its state's scale) or 2^-8 (bfloat16).  All of it counts in the weighted sum, all but the last in the sum of weights too, which multiplies
    Y.  The weighted sum adds 2^-23 of itself for each of its steps of 16 keys.  Y is rounded once, 2^-8."""
    d, group = case.d, case.P1.shape[1] // case.q8[0].shape[1 if case.layout == BHTD else 2]
    P1 = case.P1.double().numpy()
    starts = case.starts.numpy()
    order = (0, 1, 2) if case.layout == BHTD else (0, 2, 1)
    scales = case.q8[2].double().permute(*order, 3).numpy()
    K, V = (p.permute(*order, 3).numpy() for p in case.pools)  # [pages, G, page, d]
    for n in only:
        r = int(np.searchsorted(starts, n, side="right")) - 1
        c, f = case.rows[r]
        t, few = n - int(starts[r]), f * group <= 16
        i = c + t
        ids = case.table[r, : -(-(i + 1) // case.page)].long().numpy()
        for h in range(P1.shape[1]):
            g = h // group
            k, v, s = (x[ids, g].reshape(-1, x.shape[-1])[: i + 1] for x in (K, V, scales))
            p = P1[n, h]
            half = k @ p / (2 * math.sqrt(d))
            self_ = np.arange(i + 1) == i
            with np.errstate(over="ignore"):
                R = np.where(self_, 0.5 + 0.5 * np.tanh(half / case.tau) + case.lam * math.log(i + 1),
                             half * (1 + np.tanh(half)))
            e = 9 * 2.0 ** -23 * (np.abs(k) @ np.abs(p) + (1152 * s[:, 0] * np.abs(p).sum() if few else 0))
            e += 2.0 ** -25 * np.abs(p).max() * np.abs(k).sum(1) if few else 0
            e = e / (2 * math.sqrt(d)) * np.where(self_, 0.5 / case.tau, 2.2)  # |dR/d(U/2)|
            e += 2.0 ** -10.9 * np.where(self_, 0.5, np.abs(half * np.tanh(half)))
            top = float((R + np.log(np.maximum(s[:, 1], 2.0 ** -64)) if few else R).max())
            e += 6 * 2.0 ** -24 * np.maximum(np.abs(R), abs(top))
            e = np.expm1(e)
            w = np.exp(R - R.max())
            w /= w.sum()
            Y = w @ v
            u = 2.0 ** -11 if few else 2.0 ** -8
            bound = 2.0 ** -8 * np.abs(Y) + 1.01 * ((w * (e + u + (i + 1) / 16 * 2.0 ** -23)) @ np.abs(v) + np.abs(Y) * (w @ e))
            if few:
                bound = bound + 2.0 ** -32 * (w * s[:, 1]).max() * (np.abs(v) / s[:, 1:]).sum(0)
            yield n, h, Y, bound


def check_rows(case, Y, only, worst=5.0):
    """Every value within its row's bound, which is a small part of the row: `worst` times below its largest value, so
    that no row passes as zeros or as another one."""
    got = Y.double().numpy()
    for n, h, want, bound in rows_of(case, only):
        off = np.abs(got[n, h] - want)
        assert (off <= bound).all(), (n, h, float((off / bound).max()))
        assert bound.max() * worst <= np.abs(want).max(), (n, h, float(bound.max()), float(np.abs(want).max()))


MORE = {
    "drafted_g4_d128": dict(rows=[(3000, 3), (700, 4), (5000, 2)], H=8, G=2, d=128, page=64),
    "drafted_g2_d80": dict(rows=[(2500, 8), (900, 5), (40, 7)], H=4, G=2, d=80, page=32, layout=BTHD),
    "drafted_g2_d64": dict(rows=[(6000, 5), (8192, 3)], H=4, G=2, d=64, page=32),
    "drafted_d60": dict(rows=[(4000, 9), (1300, 16)], H=2, G=2, d=60, page=16),
    "prompts_d60": dict(rows=[(0, 700), (0, 40)], H=2, G=2, d=60, page=16),
    "chunk_long_d60": dict(rows=[(7000, 130)], H=2, G=2, d=60, page=16, layout=BTHD),
    "chunk_long_d80": dict(rows=[(5000, 100)], H=3, G=1, d=80, page=64),
}
CASES = {n: c for n, c in {**FWD, **LONG, **MORE}.items() if c.get("dtype") is not torch.float32}


@pytest.mark.parametrize("name", list(CASES))
def test_every_row_within_its_own_bound(name):
    case = Q8Case(**CASES[name])
    Y, _ = case.run()
    assert rb.relation_check_device_status() == 0
    ends = case.starts[1:].tolist()
    some = np.random.default_rng(2).integers(0, ends[-1], 24).tolist()
    check_rows(case, Y, sorted({*some, 0, *(e - 1 for e in ends if e > 0)}))
