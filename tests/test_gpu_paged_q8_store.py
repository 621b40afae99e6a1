"""The 8-bit pages' store and reader on the GPU: whole numbers and scales against the prologue in 64 bits, what is read
against what is held, bit for bit."""
import numpy as np
import pytest
import torch

from oracle import paged as po
from relation_token_mixing_gb300 import binding as rb

pytestmark = pytest.mark.gpu
LAYOUTS = [rb.RELATION_LAYOUT_BHTD, rb.RELATION_LAYOUT_BTHD]


def _case(N, H, G, d, page, layout, seed=0, scale=1.0):
    gen = torch.Generator().manual_seed(seed)
    pages = -(-N // page) + 3
    slots = torch.randperm(pages * page, generator=gen)[:N]
    x = {k: (torch.randn(N, h, d, generator=gen) * scale).bfloat16() for k, h in (("X1", H), ("X2", G), ("I", G))}
    x["theta"] = 0.5 * torch.randn(G // 2, generator=gen)
    x["positions"] = torch.randint(0, 40000, (N,), generator=gen, dtype=torch.int32)
    return x, slots, rb.paged_pages_q8(pages, G, page, d, layout)


def _store(x, slots, pools, layout, theta=True, pairing=0, base=1e4):
    P1 = torch.empty_like(x["X1"], device="cuda")
    c = {k: t.cuda() for k, t in x.items()}
    rb.paged_store_q8(c["X1"], c["X2"], c["I"], c["theta"] if theta else None, pairing, base, c["positions"], slots.cuda(),
                      P1, *pools, layout)
    return P1


def _held(pools, slots, page, layout, d):
    """(q, scale) of both rows of each slot, on the host in 64 bits: [N, G, d] and [N, G]."""
    out = []
    for which in (0, 1):
        rows = [np.stack([po.row_of(pools[which].cpu().numpy(), int(s), g, page, layout)[:d] for g in
                          range(pools[0].shape[1 if layout == 0 else 2])]) for s in slots]
        sc = [np.stack([po.row_of(pools[2].float().cpu().numpy(), int(s), g, page, layout)[which] for g in
                        range(pools[0].shape[1 if layout == 0 else 2])]) for s in slots]
        out.append((np.array(rows, dtype=np.float64), np.array(sc, dtype=np.float64)))
    return out


def _check_rows(q, s, x):
    """q s is x to half a step.  In float32 a turned value is off by the angle's 4e-7 and three roundings, 6e-7 of the
    pair's length, sqrt(2) of the row's largest value at most, 127 steps: 1.1e-4 of a step."""
    top = np.abs(x).max(-1)
    assert (np.log2(s) % 1 == 0).all() and (top <= 127 * s * (1 + 1e-6)).all()
    assert ((63.5 * s * (1 - 1e-6) < top) | (s == 2.0 ** -126)).all()
    assert (np.abs(q) <= 127).all()
    assert (np.abs(q - x / s[..., None]) <= 0.5 + 2e-4).all()


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("N,H,G,d,page", [(1, 2, 2, 64, 16), (70, 8, 4, 48, 32), (33, 4, 4, 60, 16), (130, 10, 2, 80, 64),
                                          (41, 8, 2, 128, 256), (700, 4, 2, 64, 128)])
def test_rows_and_scales(N, H, G, d, page, layout):
    x, slots, pools = _case(N, H, G, d, page, layout, seed=N)
    P1 = _store(x, slots, pools, layout)
    torch.cuda.synchronize()
    assert rb.relation_check_device_status() == 0
    wide = [np.zeros((*pools[0].shape[:3], d)) for _ in range(2)]
    P1r, *rows = po.store(x["X1"].double(), x["X2"].double(), x["I"].double(), x["theta"].double().numpy(), 0, 1e4,
                          x["positions"], slots, *wide, page, layout)
    assert (np.abs(P1.double().cpu().numpy() - P1r) <= 2.0 ** -8 * np.abs(P1r) + 6e-7 * 6).all()
    for (q, s), ref in zip(_held(pools, slots, page, layout, d), rows):
        _check_rows(q, s, np.stack([np.stack([po.row_of(ref, int(n), g, page, layout) for g in range(G)]) for n in slots]))
    # what is read is what is held, exactly; a negative slot reads as zeros
    some = torch.cat([slots[:5], torch.tensor([-1])])
    got = rb.paged_read_q8(some.cuda(), *pools, d, layout=layout)
    for x_, (q, s) in zip(got, _held(pools, some[:-1], page, layout, d)):
        assert (x_[:-1].double().cpu().numpy() == q * s[..., None]).all() and (x_[-1] == 0).all()


@pytest.mark.parametrize("theta,pairing,base", [(False, 0, 1e4), (True, 1, 1e4), (True, 0, 0.0)])
def test_mixing_and_rotation(theta, pairing, base):
    N, G, d, page = 20, 4, 64, 16
    x, slots, pools = _case(N, G, G, d, page, 0, seed=5)
    P1 = _store(x, slots, pools, 0, theta, pairing, base)
    torch.cuda.synchronize()
    wide = [np.zeros((*pools[0].shape[:3], d)) for _ in range(2)]
    P1r, *rows = po.store(x["X1"].double(), x["X2"].double(), x["I"].double(),
                          x["theta"].double().numpy() if theta else None, pairing, base, x["positions"], slots, *wide, page, 0)
    assert (np.abs(P1.double().cpu().numpy() - P1r) <= 2.0 ** -8 * np.abs(P1r) + 6e-7 * 6).all()
    for (q, s), ref in zip(_held(pools, slots, page, 0, d), rows):
        _check_rows(q, s, np.stack([np.stack([po.row_of(ref, int(n), g, page, 0) for g in range(G)]) for n in slots]))


@pytest.mark.parametrize("scale", [0.0, 1e-38, 3e-20, 1e20, 2.0 ** 122])
def test_small_and_large_rows(scale):
    """Rows unturned, so that the reference is exact: zeros, values next to the least and the greatest of bf16."""
    x, slots, pools = _case(40, 2, 2, 60, 16, 0, seed=1, scale=scale)
    _store(x, slots, pools, 0, theta=False, base=0.0)
    for (q, s), k in zip(_held(pools, slots, 16, 0, 60), ("X2", "I")):
        _check_rows(q, s, x[k].double().numpy())
    got = rb.paged_read_q8(slots.cuda(), *pools, 60)
    for x_, (q, s) in zip(got, _held(pools, slots, 16, 0, 60)):
        assert (x_.double().cpu().numpy() == q * s[..., None]).all()


def test_scales_at_their_border():
    """127 2^k is held at the scale 2^k, the next bf16 value above at twice that."""
    x, slots, pools = _case(3, 1, 1, 64, 16, 0)
    x["I"] = torch.zeros_like(x["I"])
    x["I"][:, 0, 5] = torch.tensor([127.0, 127.5, -127.0 * 2.0 ** -20])
    _store(x, slots, pools, 0, theta=False, base=0.0)
    (_, _), (q, s) = _held(pools, slots, 16, 0, 64)
    assert s[:, 0].tolist() == [1.0, 2.0, 2.0 ** -20] and q[:, 0, 5].tolist() == [127.0, 64.0, -127.0]


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_rows_that_are_not_finite_read_as_nan(value):
    x, slots, pools = _case(4, 2, 2, 64, 16, 0)
    x["X2"][1, 0, 3] = value
    x["I"][2, 1, 60] = value
    _store(x, slots, pools, 0, theta=False, base=0.0)
    P2, I = rb.paged_read_q8(slots.cuda(), *pools, 64)
    torch.cuda.synchronize()
    assert rb.relation_check_device_status() == 0
    for rows, n, g in ((P2, 1, 0), (I, 2, 1)):
        bad = torch.zeros(4, 2, dtype=torch.bool)
        bad[n, g] = True
        assert torch.equal(torch.isnan(rows).all(-1).cpu(), bad) and torch.equal(torch.isnan(rows).any(-1).cpu(), bad)


def test_slots_that_are_not_there():
    x, slots, pools = _case(20, 2, 2, 64, 16, 0, seed=2)
    slots[3], slots[7] = -1, pools[0].shape[0] * 16
    before = [p.clone() for p in pools]
    P1 = _store(x, slots, pools, 0)
    torch.cuda.synchronize()
    assert rb.relation_check_device_status() == 1 and rb.relation_check_device_status() == 0
    assert torch.isfinite(P1).all()
    written = torch.zeros(pools[0].shape[0] * 16, dtype=torch.bool)
    keep = [int(s) for n, s in enumerate(slots) if n not in (3, 7)]
    written[keep] = True
    rest = (~written).view(-1, 16).nonzero()
    for p, b in zip(pools, before):  # nothing else is touched
        assert torch.equal(p[rest[:, 0], :, rest[:, 1]], b[rest[:, 0], :, rest[:, 1]])
    P2, I = rb.paged_read_q8(slots.cuda(), *pools, 64)
    torch.cuda.synchronize()
    assert rb.relation_check_device_status() == 1
    assert (P2[[3, 7]] == 0).all() and (I[[3, 7]] == 0).all() and (P2[0] != 0).any()


def test_no_tokens_and_another_stream():
    x, slots, pools = _case(64, 4, 2, 80, 32, 0, seed=9)
    P1 = _store(x, slots, pools, 0)
    want = rb.paged_read_q8(slots.cuda(), *pools, 80)
    again = rb.paged_pages_q8(pools[0].shape[0], 2, 32, 80)
    c = {k: t.cuda() for k, t in x.items()}
    s, out = slots.cuda(), torch.empty_like(P1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    rb.paged_store_q8(c["X1"], c["X2"], c["I"], c["theta"], 0, 1e4, c["positions"], s, out, *again, stream=side)
    got = rb.paged_read_q8(s, *again, 80, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert torch.equal(out, P1) and all(torch.equal(a, b) for a, b in zip(got, want))
    none = torch.empty(0, dtype=torch.int64, device="cuda")
    assert rb.paged_read_q8(none, *pools, 80)[0].shape == (0, 2, 80)
    assert rb.relation_check_device_status() == 0
