"""Pins of the paged Relation Cache oracle (CPU), and the host-side checks of its entry points."""
import ctypes

import numpy as np
import pytest
import torch

import oracle
from oracle import paged as po
from oracle import prologue
from relation_token_mixing_gb300 import binding as rb

A = 0x100000  # fake, 16-byte aligned addresses 1 MiB apart


def test_plan_by_hand():
    """Pages of 16: request 0 holds one page (9 tokens) and takes 8 more tokens (one new page), request 1 has
    none, request 2 fills its page exactly and takes one token, request 3 starts from nothing."""
    table = [[5, -1, -1], [7, -1, -1], [4, -1, -1], [-1, -1, -1]]
    t, starts, slots, pos, used = po.plan([9, 3, 16, 0], [8, 0, 1, 17], [2, 0, 6], table, 8, 16, 28)
    assert t.tolist() == [[5, 2, -1], [7, -1, -1], [4, 0, -1], [6, -1, -1]]
    assert starts.tolist() == [0, 8, 8, 9, 26]
    assert used == 4  # one more than the free list holds
    assert slots[:8].tolist() == [5 * 16 + k for k in range(9, 16)] + [2 * 16]
    assert slots[8] == 0 and pos[8] == 16
    assert slots[9:25].tolist() == [6 * 16 + k for k in range(16)]
    assert slots[25] == -1 and pos[25] == 16  # the page that the free list could not serve
    assert slots[26:].tolist() == [-1, -1] and pos[26:].tolist() == [0, 0]


@pytest.mark.parametrize("layout", [po.BHTD, po.BTHD])
@pytest.mark.parametrize("group", [1, 3])
def test_forward_equals_the_operator_over_contiguous_tokens(layout, group):
    """Chunked, shuffled pages give the rows of the causal operator (grouped heads: the shared rows repeated)."""
    rng = np.random.default_rng(1)
    G, d, page, total, cached = 2, 8, 16, 41, 23
    H = G * group
    P1, K, V = rng.standard_normal((3, 1, H, total, d))
    K, V = K[:, :G], V[:, :G]
    rep = [np.repeat(x, group, axis=1) for x in (K, V)]
    Yr, Lr = oracle.fwd(P1, rep[0], rep[1], 0.7, 0.5, True)
    table = np.array([[3, 0, 4]])
    shape = (5, G, page, d) if layout == po.BHTD else (5, page, G, d)
    pools = [np.full(shape, np.nan) for _ in range(2)]
    for pool, x in zip(pools, (K, V)):
        for j in range(total):
            for g in range(G):
                po.row_of(pool, int(table[0, j // page]) * page + j % page, g, page, layout)[:] = x[0, g, j]
    Y, L = po.fwd(P1[0, :, cached:].transpose(1, 0, 2), *pools, table, [0, total - cached], [cached], 0.7, 0.5, page,
                  layout)
    np.testing.assert_allclose(Y, np.asarray(Yr)[0, :, cached:].transpose(1, 0, 2), atol=1e-12)
    np.testing.assert_allclose(L, np.asarray(Lr)[0, :, cached:].T, atol=1e-12)


@pytest.mark.parametrize("pairing", [0, 1])
def test_store_equals_the_prologue(pairing):
    rng = np.random.default_rng(2)
    N, H, G, d, page = 11, 4, 4, 6, 16
    X1, X2, I = rng.standard_normal((3, N, H, d))
    theta = rng.standard_normal(G // 2)
    pools = np.zeros((2, 1, G, page, d))
    P1, P2p, Ip = po.store(X1, X2, I, theta, pairing, 1e4, np.arange(5, 5 + N), np.arange(N), *pools, page, po.BHTD)
    heads_first = lambda x: x.transpose(1, 0, 2)[None]  # noqa: E731
    np.testing.assert_allclose(heads_first(P1), prologue.rope(heads_first(X1), 1e4, [5]), atol=1e-13)
    np.testing.assert_allclose(P2p[:, :, :N], prologue.rope(heads_first(X2), 1e4, [5]), atol=1e-13)
    np.testing.assert_allclose(Ip[:, :, :N], prologue.givens(heads_first(I), theta, pairing), atol=1e-13)


def _prob(**kw):
    base = dict(R=4, N=32, H=8, G=4, d_h=64, pages=16, page_size=16, table_width=8, dtype=rb.RELATION_BF16, tau_S=1.0,
                lam=0.5, layout=0)
    base.update(kw)
    return rb.Paged(*(base[f[0]] for f in rb.Paged._fields_))


def _plan(p, **kw):
    a = dict(cached=A, fresh=2 * A, free=3 * A, count=4, table=4 * A, starts=5 * A, slots=6 * A, pos=7 * A, used=8 * A)
    a.update(kw)
    return rb.load().relation_paged_plan(ctypes.byref(p), a["cached"], a["fresh"], a["free"], a["count"], a["table"],
                                         a["starts"], a["slots"], a["pos"], a["used"], None)


def _store(p, **kw):
    a = dict(X1=A, X2=2 * A, I=3 * A, theta=4 * A, pairing=0, base=1e4, pos=5 * A, slots=6 * A, P1=7 * A, P2p=8 * A,
             Ip=10 * A)
    a.update(kw)
    return rb.load().relation_paged_store(ctypes.byref(p), a["X1"], a["X2"], a["I"], a["theta"], a["pairing"],
                                          a["base"], a["pos"], a["slots"], a["P1"], a["P2p"], a["Ip"], None)


def _fwd(p, **kw):
    a = dict(P1=A, P2p=2 * A, Ip=4 * A, table=6 * A, starts=7 * A, cached=8 * A, max_fresh=1, Y=9 * A, L=10 * A,
             ws=64 * A, n=1 << 40)
    a.update(kw)
    return rb.load().relation_paged_fwd(ctypes.byref(p), a["P1"], a["P2p"], a["Ip"], a["table"], a["starts"],
                                        a["cached"], a["max_fresh"], a["Y"], a["L"], a["ws"], a["n"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(R=0), 1), (dict(R=(1 << 20) + 1), 1), (dict(N=-1), 1), (dict(N=1 << 31), 1), (dict(H=0), 1),
    (dict(H=1025, G=1), 1), (dict(G=3), 1), (dict(G=16), 1), (dict(G=0), 1), (dict(d_h=0), 1), (dict(pages=0), 1),
    (dict(table_width=0), 1), (dict(table_width=1 << 27), 1), (dict(dtype=5), 1), (dict(layout=2), 1),
    (dict(tau_S=0.0), 1), (dict(tau_S=float("nan")), 1), (dict(lam=float("inf")), 1), (dict(pages=1 << 30), 1),
    (dict(page_size=8), 2), (dict(page_size=24), 2), (dict(page_size=512), 2), (dict(d_h=32), 2), (dict(d_h=72), 2)])
def test_problem_checks(kw, code):
    p = _prob(**kw)
    assert _plan(p) == code and _store(p) == code and _fwd(p) == code
    assert rb.relation_paged_workspace_bytes(p, 1) == 0


def test_pointer_checks():
    """Missing, misaligned and overlapping pointers are refused before the GPU is touched."""
    p = _prob()
    for k in ("cached", "fresh", "free", "table", "starts", "slots", "pos", "used"):
        assert _plan(p, **{k: None}) == 1, k
    assert _plan(p, cached=A + 2) == 3 and _plan(p, slots=6 * A + 8) == 3 and _plan(p, table=4 * A + 4) == 3
    assert _plan(p, starts=A + 4) == 1 and _plan(p, pos=6 * A + 16) == 1 and _plan(p, count=1 << 31) == 1
    for k in ("X1", "X2", "I", "pos", "slots", "P1", "P2p", "Ip"):
        assert _store(p, **{k: None}) == 1, k
    assert _store(p, X1=A + 8) == 3 and _store(p, theta=4 * A + 2) == 3 and _store(p, Ip=10 * A + 4) == 3
    assert _store(p, P1=A) == 1 and _store(p, Ip=8 * A + 16) == 1
    assert _store(p, pairing=2) == 1 and _store(p, base=float("nan")) == 1
    assert _store(_prob(H=8, G=1)) == 1  # mixing needs pairs of cache heads
    for k in ("P1", "P2p", "Ip", "table", "starts", "cached", "Y", "ws"):
        assert _fwd(p, **{k: None}) == 1, k
    assert _fwd(p, P1=A + 8) == 3 and _fwd(p, L=10 * A + 2) == 3 and _fwd(p, ws=64 * A + 8) == 3
    assert _fwd(p, max_fresh=-1) == 1
    assert _fwd(_prob(R=8193)) == 2


def test_struct_matches_the_header():
    import os
    import re
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "relation.h")
    body = re.search(r"typedef struct \{([^}]*)\} relation_paged_t;", open(path).read()).group(1)
    body = re.sub(r"/\*.*?\*/", "", body, flags=re.S)
    names = [n.strip() for decl in body.split(";") if decl.strip() for n in decl.strip().split(None, 1)[1].split(",")]
    assert [{"lam": "lambda"}.get(f[0], f[0]) for f in rb.Paged._fields_] == names
    assert ctypes.sizeof(rb.Paged) == 8 * 8 + 4 * 4


def test_binding_refuses_mismatched_tensors():
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    with pytest.raises(ValueError, match="slots"):
        rb.paged_plan(i32(2), i32(2), None, i32(2, 4), 8, 16, i32(3), i32(5), i32(5), i32(1))
    with pytest.raises(ValueError, match="starts"):
        rb.paged_plan(i32(2), i32(2), None, i32(2, 4), 8, 16, i32(2), i32(5).long(), i32(5), i32(1))
    with pytest.raises(ValueError, match="rows of 60"):
        rb.paged_fwd(bf(3, 4, 60), bf(8, 2, 16, 60), bf(8, 2, 16, 60), i32(1, 4), i32(2), i32(1), 0, 1.0, 0.5)
    with pytest.raises(ValueError, match="dtype"):
        rb.paged_fwd(bf(3, 4, 64), bf(8, 2, 16, 64).float(), bf(8, 2, 16, 64), i32(1, 4), i32(2), i32(1), 0, 1.0, 0.5)
    with pytest.raises(ValueError, match="starts"):
        rb.paged_fwd(bf(3, 4, 64), bf(8, 2, 16, 64), bf(8, 2, 16, 64), i32(1, 4), i32(3), i32(1), 0, 1.0, 0.5)
    with pytest.raises(ValueError, match="X1, P1"):
        rb.paged_store(bf(3, 4, 64), bf(3, 4, 64), bf(3, 2, 64), None, 0, 1e4, i32(3), i32(3).long(), bf(3, 4, 64),
                       bf(8, 2, 16, 64), bf(8, 2, 16, 64))
