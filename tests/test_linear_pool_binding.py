"""What Linear Relation over a pool of states refuses on the host (CPU; every call here fails its checks)."""
import ctypes

import numpy as np
import pytest
import torch

from linear_pool_cases import inputs, packed, reference
from relation_token_mixing_gb300 import binding as rb

A = 1 << 24  # fake addresses 16 MB apart, aligned


def _prob(**kw):
    a = dict(R=3, N=40, H=2, d_h=64, states=4, dtype=rb.RELATION_BF16, tau_S=2.0) | kw
    return rb.LinearPacked(a["R"], a["N"], a["H"], a["d_h"], a["states"], a["dtype"], a["tau_S"])


NAMES = ("P1", "P2", "I", "G", "A_log", "dt_bias", "starts", "states", "slots_in", "slots_out", "Y", "ws")


def _call(prob, step=False, max_fresh=10, nbytes=1 << 20, **kw):
    a = {k: (n + 1) * A for n, k in enumerate(NAMES)} | kw
    lib = rb.load()
    if step:
        return lib.relation_linear_step(ctypes.byref(prob), a["P1"], a["P2"], a["I"], a["G"], a["A_log"], a["dt_bias"],
                                        a["states"], a["slots_in"], a["slots_out"], a["Y"], None)
    return lib.relation_linear_packed_fwd(ctypes.byref(prob), a["P1"], a["P2"], a["I"], a["G"], a["A_log"],
                                          a["dt_bias"], a["starts"], max_fresh, a["states"], a["slots_in"],
                                          a["slots_out"], a["Y"], a["ws"], nbytes, None)


def test_struct_matches_the_header():
    assert [f[0] for f in rb.LinearPacked._fields_] == ["R", "N", "H", "d_h", "states", "dtype", "tau_S"]
    assert ctypes.sizeof(rb.LinearPacked) == 5 * 8 + 2 * 4


@pytest.mark.parametrize("kw,code", [(dict(R=0), 1), (dict(R=(1 << 20) + 1), 1), (dict(N=-1), 1), (dict(N=1 << 31), 1),
                                     (dict(H=0), 1), (dict(H=1025), 1), (dict(states=0), 1), (dict(states=1 << 31), 1),
                                     (dict(dtype=5), 1), (dict(tau_S=0.0), 1), (dict(tau_S=float("nan")), 1),
                                     (dict(d_h=0), 1), (dict(d_h=80), 2), (dict(d_h=128), 2),
                                     (dict(dtype=rb.RELATION_F32), 2), (dict(states=1 << 30, H=1024), 1),
                                     (dict(N=(1 << 31) - 1, H=1024), 1)])
def test_problems_are_refused(kw, code):
    for step in (False, True):
        assert _call(_prob(**kw), step) == code
    assert rb.relation_linear_packed_workspace_bytes(_prob(**kw), 0) == 0


@pytest.mark.parametrize("kw,code", [({k: None}, 1) for k in NAMES if k not in ("ws", "A_log", "dt_bias")] +
                         [({"A_log": None}, 1), ({"dt_bias": None}, 1)] +
                         [({k: A * (n + 1) + (2 if k in ("A_log", "dt_bias", "starts", "slots_in", "slots_out") else 8)}, 3)
                          for n, k in enumerate(NAMES)])
def test_pointers_are_refused(kw, code):
    assert _call(_prob(), **kw) == code
    if "starts" not in kw and "ws" not in kw:
        assert _call(_prob(), True, **kw) == code


def test_sizes_are_refused():
    assert _call(_prob(), max_fresh=-1) == 1
    assert _call(_prob(N=2), True) == 1  # fewer rows than requests
    assert rb.relation_linear_packed_workspace_bytes(_prob(), -1) == 0


def _t(*s, dtype=torch.bfloat16):
    return torch.zeros(*s, dtype=dtype)


@pytest.mark.parametrize("kw", [dict(P2=_t(5, 2, 60)), dict(I=_t(5, 2, 64, dtype=torch.float32)),
                                dict(G=_t(5, 2, 64)), dict(states=_t(3, 2, 64, 60, dtype=torch.float32)),
                                dict(states=_t(3, 2, 64, 64)), dict(slots_in=_t(2, dtype=torch.int64)),
                                dict(slots_out=_t(3, dtype=torch.int32)), dict(A_log=_t(2, 64, dtype=torch.float32)),
                                dict(A_log=_t(2, 64), dt_bias=_t(2, 64)), dict(starts=_t(2, dtype=torch.int32)),
                                dict(starts=_t(3, dtype=torch.int64)), dict(P1=_t(5, 2, 64, dtype=torch.float16)),
                                dict(Y=_t(5, 2, 60))])
def test_the_wrapper_refuses_shapes_and_types(kw):
    a = dict(P1=_t(5, 2, 64), P2=_t(5, 2, 64), I=_t(5, 2, 64), G=_t(5, 2, 64, dtype=torch.float32),
             starts=_t(3, dtype=torch.int32), states=_t(3, 2, 64, 64, dtype=torch.float32),
             slots_in=_t(2, dtype=torch.int32), slots_out=_t(2, dtype=torch.int32), A_log=None, dt_bias=None, Y=None) | kw
    if a["Y"] is None:
        a["Y"] = _t(5, 2, 64)
    Y = a.pop("Y")
    with pytest.raises(ValueError):
        packed(a, Y=Y)


def test_the_wrapper_refuses_host_tensors():
    x = inputs([2, 1], 2, 64)
    with pytest.raises(ValueError, match="CUDA"):
        packed(x, Y=torch.empty_like(x["P1"]), workspace=torch.empty(16, dtype=torch.uint8))


def test_oracle_in_one_piece_and_in_two():
    """The recurrence of a request, and of its two halves from slot to slot, against the dense oracle."""
    from oracle import linear as dense

    x = inputs([12], 2, 48, slots=([-1], [0]), seed=1)
    (Y, S), (_, Sa) = reference(x)
    heads = {k: x[k].double().numpy().transpose(1, 0, 2)[None] for k in ("P1", "P2", "I", "G")}
    Yd, Cd = dense.fwd(heads["P1"], heads["P2"], heads["I"], heads["G"], 2.0)
    assert np.allclose(Y.transpose(1, 0, 2), Yd[0], atol=1e-12) and np.allclose(S[0], Cd[0], atol=1e-12)
    assert (np.abs(S) <= Sa + 1e-12).all()
    halves = dict(x, starts=torch.tensor([0, 7], dtype=torch.int32))
    mid = torch.from_numpy(reference(halves)[0][1])
    rest = dict(x, states=mid, slots_in=torch.tensor([0], dtype=torch.int32),
                starts=torch.tensor([7, 12], dtype=torch.int32))
    (Y2, S2), _ = reference(rest)
    assert np.allclose(Y2[7:], Y[7:], atol=1e-12) and np.allclose(S2, S, atol=1e-12)
