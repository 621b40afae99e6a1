"""Non-finite values in live rows of the paged Relation Cache, against the float64 oracle.

A NaN or infinite score makes every entry of the rows that see its key NaN, whichever pieces their history is cut
into; a NaN or infinite information state reaches its own column of the rows that see it and nothing else.  Histories
are long enough to be cut into pieces among workers, and short ones beside them are taken whole.  Where the values must
be, and where they must not, is compared exactly; finite entries keep the operator's tolerances (1e-5 and 1e-2 max |V|).
"""
import numpy as np
import pytest
import torch

from oracle import paged as po
from relation_token_mixing_gb300 import binding as rb
from test_gpu_paged import BF, BTHD, F32, Case

pytestmark = pytest.mark.gpu

CASES = {
    "decode_d64": dict(rows=[(9000, 1), (12, 1)], H=4, G=2, d=64, page=64),
    "decode_one_d128": dict(rows=[(20011, 1)], H=2, G=1, d=128, page=16),
    "few_d48": dict(rows=[(5000, 3), (700, 2)], H=4, G=2, d=48, page=32, layout=BTHD),
    "chunk_d64": dict(rows=[(6000, 70), (40, 300)], H=2, G=2, d=64, page=16),
    "chunk_d80": dict(rows=[(5000, 140), (5, 30)], H=2, G=1, d=80, page=128),
    "chunk_d128": dict(rows=[(6000, 140)], H=2, G=1, d=128, page=64, layout=BTHD),
    "mixed_d64": dict(rows=[(5000, 1), (900, 200), (3000, 4)], H=4, G=2, d=64, page=32),
    "f32_decode_d64": dict(rows=[(9000, 1), (12, 1)], H=4, G=2, d=64, page=64, dtype=F32),
    "f32_chunk_d128": dict(rows=[(4000, 70), (5, 20)], H=2, G=1, d=128, page=16, dtype=F32),
}


def _set(case, which, request, tokens, columns, value):
    """value in the given columns of cached rows of cache head 0."""
    for t in tokens:
        slot = int(case.table[request, t // case.page]) * case.page + t % case.page
        po.row_of(case.pools[which], slot, 0, case.page, case.layout)[columns] = value


def _check(case, sample):
    Y, L = case.run()
    assert rb.relation_check_device_status() == 0
    with np.errstate(invalid="ignore"):
        refY, refL = po.fwd(case.P1.double(), *(p.double().numpy() for p in case.pools), case.table.numpy(),
                            case.starts.numpy(), case.cached.numpy(), case.tau, case.lam, case.page, case.layout, sample)
    got, gotL, want = Y.double().numpy()[sample], L.double().numpy()[sample], refY[sample]
    finite = np.isfinite(want)
    np.testing.assert_array_equal(np.isfinite(got), finite)
    # what an infinite state leaves is infinite on the same side, the rest is NaN
    np.testing.assert_array_equal(np.nan_to_num(got[~finite], nan=7.0), np.nan_to_num(want[~finite], nan=7.0))
    np.testing.assert_array_equal(np.isfinite(gotL), np.isfinite(refL[sample]))
    assert np.abs(got[finite] - want[finite]).max(initial=0.0) <= (1e-5 if case.P1.dtype is F32 else 1e-2) * case.vmax
    return finite


def _sample(case):
    ends = case.starts.tolist()
    return sorted({n for a, b in zip(ends, ends[1:]) for n in (a, (a + b) // 2, b - 1) if a < b})


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("at", [0, 37, 64, 1000])
@pytest.mark.parametrize("name", list(CASES))
def test_one_non_finite_key_makes_its_rows_nan(name, at, value):
    case = Case(**CASES[name])
    at = min(at, CASES[name]["rows"][0][0] - 1)
    _set(case, 0, 0, [at], slice(2, 3), value)
    finite = _check(case, _sample(case))
    assert not finite.all() and (len(case.rows) == 1 or finite.any())


@pytest.mark.parametrize("name", list(CASES))
@pytest.mark.parametrize("first", [0, 64, 256])
def test_a_stretch_of_nan_keys(name, first):
    """Whole pieces of nothing but NaN scores: every key tile of the kernels begins at a multiple of 32, 64 or 128."""
    case = Case(**CASES[name])
    for length in (64, 128):
        _set(case, 0, 0, range(first, first + length), slice(None), float("nan"))
        _check(case, _sample(case))


@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("name", list(CASES))
def test_a_non_finite_state_stays_in_its_column(name, value):
    case = Case(**CASES[name])
    _set(case, 1, 0, [77], slice(5, 6), value)
    finite = _check(case, _sample(case))
    assert not finite.all() and finite[..., :5].all() and finite[..., 6:].all()


@pytest.mark.parametrize("name", list(CASES))
def test_a_nan_query_is_its_own(name):
    case = Case(**CASES[name])
    sample = _sample(case)
    case.P1[sample[-1], 0, 3] = float("nan")
    finite = _check(case, sample)
    assert not finite[-1, 0].any() and finite[:-1].all() and finite[-1, 1:].all()
