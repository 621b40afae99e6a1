"""What the 8-bit pages' calls refuse on the host (CPU; every call here fails its checks)."""
import ctypes

import pytest
import torch

from relation_token_mixing_gb300 import binding as rb

A = 1 << 26  # fake addresses 64 MB apart, aligned
STORE = ("X1", "X2", "I", "theta", "positions", "slots", "P1", "P2_pages", "I_pages", "scales")
READ = ("slots", "P2_pages", "I_pages", "scales", "P2", "I")
FWD = ("P1", "P2_pages", "I_pages", "scales", "block_table", "starts", "cached", "Y", "L", "ws")


def _prob(**kw):
    a = dict(R=3, N=40, H=4, G=2, d_h=64, pages=20, page_size=16, table_width=8, dtype=rb.RELATION_BF16, tau_S=2.0,
             lam=0.5, layout=rb.RELATION_LAYOUT_BHTD) | kw
    return rb.Paged(*a.values())


def _at(names, kw):
    return {k: (n + 1) * A for n, k in enumerate(names)} | kw


def _store(p, pairing=0, base=1e4, **kw):
    a = _at(STORE, kw)
    return rb.load().relation_paged_store_q8(ctypes.byref(p), a["X1"], a["X2"], a["I"], a["theta"], pairing, base,
                                             *(a[k] for k in STORE[4:]), None)


def _read(p, **kw):
    return rb.load().relation_paged_read_q8(ctypes.byref(p), *_at(READ, kw).values(), None)


def _fwd(p, max_fresh=4, nbytes=1 << 30, **kw):
    a = _at(FWD, kw)
    return rb.load().relation_paged_fwd_q8(ctypes.byref(p), *(a[k] for k in FWD[:7]), max_fresh, a["Y"], a["L"], a["ws"],
                                           nbytes, None)


@pytest.mark.parametrize("kw,code", [(dict(R=0), 1), (dict(N=-1), 1), (dict(H=3), 1), (dict(G=0), 1), (dict(pages=0), 1),
                                     (dict(page_size=48), 2), (dict(page_size=8), 2), (dict(page_size=512), 2),
                                     (dict(d_h=96), 2), (dict(d_h=0), 1), (dict(dtype=rb.RELATION_F32), 2),
                                     (dict(dtype=9), 1), (dict(layout=2), 1), (dict(tau_S=-1.0), 1)])
def test_problems_are_refused(kw, code):
    p = _prob(**kw)
    assert _store(p) == code and _read(p) == code and _fwd(p) == code
    assert rb.relation_paged_q8_workspace_bytes(p, 4) == 0


@pytest.mark.parametrize("call,names,free", [(_store, STORE, ("theta",)), (_read, READ, ()), (_fwd, FWD, ("L",))])
def test_pointers_are_refused(call, names, free):
    for n, k in enumerate(names):
        if k not in free:
            assert call(_prob(), **{k: None}) == 1, k
        assert call(_prob(), **{k: (n + 1) * A + 2}) == 3, k


def test_other_arguments_are_refused():
    assert _store(_prob(), pairing=2) == 1 and _store(_prob(), base=float("nan")) == 1
    assert _store(_prob(H=3, G=3)) == 1  # mixing pairs the cache heads
    assert _fwd(_prob(), max_fresh=-1) == 1
    assert _fwd(_prob(R=8193)) == 2
    assert _fwd(_prob(H=1024, G=1, N=1 << 22), max_fresh=1 << 21) == 2


def test_overlaps_are_refused():
    """(Read's checks come before any device call; the forward's need the device's workspace size.)"""
    assert _store(_prob(), P1=A) == 1 and _store(_prob(), scales=8 * A + 64) == 1
    assert _read(_prob(), P2=2 * A) == 1 and _read(_prob(), I=5 * A + 16) == 1


def test_nothing_to_do():
    p = _prob(N=0)
    assert _store(p, X1=None) == 0 and _read(p, P2=None) == 0 and _fwd(p, P1=None) == 0


def _pools(layout=0, d=64, row=None):
    shape = (20, 2, 16) if layout == 0 else (20, 16, 2)
    row = rb.paged_row_q8(d) if row is None else row
    return [torch.zeros(*shape, row, dtype=torch.int8) for _ in range(2)] + [torch.zeros(*shape, 2, dtype=torch.bfloat16)]


def _b(*s, dtype=torch.bfloat16):
    return torch.zeros(*s, dtype=dtype)


I32, I64 = torch.int32, torch.int64


@pytest.mark.parametrize("change", [
    dict(pools=_pools(row=80)), dict(pools=[x.float() for x in _pools()]), dict(pools=_pools()[:2] + [_b(20, 2, 16)]),
    dict(pools=_pools()[:2] + [_b(20, 2, 16, 2, dtype=torch.float32)]), dict(layout=3), dict(P1=_b(5, 4, 60)),
    dict(P1=_b(5, 4, 64, dtype=torch.float32)), dict(table=_b(3, 8, dtype=I64)), dict(starts=_b(3, dtype=I32)),
    dict(cached=_b(2, dtype=I32)), dict(L=_b(5, 4)), dict(Y=_b(5, 4, 64, dtype=torch.float32))])
def test_the_forward_wrapper_refuses_shapes_and_types(change):
    a = dict(pools=_pools(), layout=0, P1=_b(5, 4, 64), table=_b(3, 8, dtype=I32), starts=_b(4, dtype=I32),
             cached=_b(3, dtype=I32), L=None, Y=_b(5, 4, 64)) | change
    with pytest.raises(ValueError):
        rb.paged_fwd_q8(a["P1"], *a["pools"], a["table"], a["starts"], a["cached"], 2, 2.0, 0.5, a["Y"], a["L"],
                        torch.zeros(16, dtype=torch.uint8), a["layout"])


@pytest.mark.parametrize("change", [
    dict(X2=_b(5, 4, 64)), dict(I=_b(4, 2, 64)), dict(P1=_b(5, 2, 64)), dict(X1=_b(5, 4, 64, dtype=torch.float32)),
    dict(theta=_b(1)), dict(theta=_b(2, dtype=torch.float32)), dict(positions=_b(5, dtype=I64)),
    dict(slots=_b(5, dtype=I32)), dict(slots=_b(4, dtype=I64))])
def test_the_store_wrapper_refuses_shapes_and_types(change):
    a = dict(X1=_b(5, 4, 64), X2=_b(5, 2, 64), I=_b(5, 2, 64), theta=None, positions=_b(5, dtype=I32),
             slots=_b(5, dtype=I64), P1=_b(5, 4, 64)) | change
    with pytest.raises(ValueError):
        rb.paged_store_q8(a["X1"], a["X2"], a["I"], a["theta"], 0, 1e4, a["positions"], a["slots"], a["P1"], *_pools())


@pytest.mark.parametrize("slots,P2", [(_b(5, dtype=I32), None), (_b(5, dtype=I64), _b(5, 2, 60)),
                                      (_b(5, dtype=I64), _b(5, 2, 64, dtype=torch.float32))])
def test_the_read_wrapper_refuses_shapes_and_types(slots, P2):
    with pytest.raises(ValueError):
        rb.paged_read_q8(slots, *_pools(), 64, P2, _b(5, 2, 64))


def test_pools_of_every_width():
    for layout in (0, 1):
        for d, row in ((48, 48), (60, 64), (64, 64), (80, 80), (128, 128)):
            P2, I, scales = rb.paged_pages_q8(3, 2, 16, d, layout, device="cpu")
            assert P2.shape == I.shape and P2.shape[3] == row and scales.shape == (*P2.shape[:3], 2)
            assert P2.shape[:3] == ((3, 2, 16) if layout == 0 else (3, 16, 2))
