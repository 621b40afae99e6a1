"""The forward over 8-bit pages on the GPU against the oracle over what the pages stand for, at the bf16 path's
tolerances (the operands are exact in both, the weights' rounding the same or finer).

Slots that hold no token have a NaN scale and whole numbers of any kind, so have the rows' paddings; block-table entries
past a request's pages are far out of range, workspaces start as NaN and rows outside the requests keep a sentinel."""
import numpy as np
import pytest
import torch

from paged_q8_cases import Q8Case
from relation_token_mixing_gb300 import binding as rb
from test_gpu_paged import FWD, LONG

pytestmark = pytest.mark.gpu
NAMES = [n for n in FWD if not n.startswith("f32")]


@pytest.mark.parametrize("name", NAMES)
def test_forward(name):
    case = Q8Case(**FWD[name], extra=3)
    Y, L = case.run()
    assert rb.relation_check_device_status() == 0
    case.check(Y, L)


@pytest.mark.parametrize("name", [n for n in LONG if "f32" not in n])
def test_forward_over_long_pieces(name):
    case = Q8Case(**LONG[name], extra=1)
    Y, L = case.run()
    assert rb.relation_check_device_status() == 0
    assert torch.isfinite(Y[: int(case.starts[-1])].float()).all()
    ends = case.starts[1:].tolist()
    case.check(Y, L, only=sorted({*np.random.default_rng(1).integers(0, ends[-1], 12).tolist(), 0, *(e - 1 for e in ends)}))


@pytest.mark.parametrize("name", ["decode_edges_d64", "few_rows_d128", "mixed", "chunk_g3_d80"])
@pytest.mark.parametrize("spread", [3, 20])
def test_rows_of_very_different_sizes(name, spread):
    """States of a token times a power of two: the weights follow the scales, the sum does not."""
    case = Q8Case(**FWD[name], spread=spread)
    Y, L = case.run()
    assert rb.relation_check_device_status() == 0
    case.check(Y, L)


def _alone(rows, H, G, d, **kw):
    """A case whose I~ rows are the caller's to set: (case, set) with set(tensor of the pool's shape)."""
    case = Q8Case(rows=rows, H=H, G=G, d=d, **kw)

    def put(q, scale):
        k, v, s = case.q8
        s = s.clone()
        s[..., 1] = torch.where(torch.isnan(s[..., 1].float()), s[..., 1], torch.as_tensor(scale).to(s.dtype))
        case.q8 = k, (v if q is None else torch.full_like(v, q)), s
        case.pools = case.pools[0], case.q8[1][..., :d].double() * s[..., 1:].double()
        live = case.pools[1][torch.isfinite(case.pools[1])]
        case.vmax = float(live.abs().max())
        return case

    return put


@pytest.mark.parametrize("rows", [[(90, 2), (0, 1)], [(90, 40)]])
@pytest.mark.parametrize("exponent", [-126, -90, -64, -20, 20, 60, 110])
def test_scales_from_the_least_to_large_ones(rows, exponent):
    """Every I~ row at one scale.  Below 2^-64 the weights' products leave float16 where there are few rows: what is
    lost of a row is below 2^-64 max|q| then, so those are compared absolutely."""
    case = _alone(rows, 4, 2, 64)(None, 2.0 ** exponent)
    Y, L = case.run()
    assert rb.relation_check_device_status() == 0
    if exponent < -64:
        case.vmax = max(case.vmax, 2.0 ** -64 * 127)
    case.check(Y, L)


@pytest.mark.parametrize("rows", [[(90, 2)], [(90, 40)]])
def test_zero_states(rows):
    case = _alone(rows, 2, 2, 64)(0, 2.0 ** -126)
    Y, L = case.run()
    n = int(case.starts[-1])
    assert (Y[:n] == 0).all()
    case.vmax = 1.0
    case.check(Y, L)


@pytest.mark.parametrize("factor", [2.0 ** -30, 2.0 ** 30])
@pytest.mark.parametrize("name", ["decode_edges_g2_d64", "chunk_g2_d60"])
def test_queries_of_very_different_sizes(name, factor):
    """Every other head's queries times a power of two, so that a group's rows differ by 2^30 (scores of nothing, and
    of 0 or very large ones)."""
    case = Q8Case(**FWD[name])
    case.P1 = case.P1.clone()
    case.P1[:, ::2] *= factor
    Y, L = case.run()
    assert rb.relation_check_device_status() == 0
    case.check(Y, L)


@pytest.mark.parametrize("which", ["key", "state"])
@pytest.mark.parametrize("rows,first", [([(70, 2), (40, 1)], 30), ([(200, 40)], 150)])
def test_a_row_that_was_not_finite_makes_the_rows_that_see_it_nan(which, rows, first):
    """One token's scale is NaN: the request's new tokens see it and are NaN, other requests' are not."""
    case = Q8Case(rows=rows, H=2, G=2, d=64)
    page = int(case.table[0, first // case.page])
    k, v, s = case.q8
    assert case.layout == rb.RELATION_LAYOUT_BHTD
    s[page, :, first % case.page, 0 if which == "key" else 1] = float("nan")
    Y, L = case.run()
    assert rb.relation_check_device_status() == 0
    hi = int(case.starts[1])
    assert torch.isnan(Y[:hi].float()).all()
    if which == "key":
        assert torch.isnan(L[:hi]).all()
    assert torch.isfinite(Y[hi: int(case.starts[-1])].float()).all()


@pytest.mark.parametrize("name", ["mixed", "mixed_d128", "few_rows", "decode_long", "chunk_d64"])
def test_the_same_from_run_to_run(name):
    case = Q8Case(**FWD[name])
    (Y, L), (Y2, L2) = case.run(), case.run()
    assert torch.equal(Y, Y2) and torch.equal(L, L2)


@pytest.mark.parametrize("name", ["mixed", "decode_edges_d64"])
def test_without_a_known_bound_on_a_stream_of_its_own(name):
    case = Q8Case(**FWD[name], first=5, extra=2)
    Y, L = case.run(max_fresh=0, stream=torch.cuda.Stream())
    assert rb.relation_check_device_status() == 0
    case.check(Y, L)


def test_what_cannot_be_followed_is_skipped_and_reported():
    rows = [(100, 1), (50, 40), (20, 2), (300, 60)]
    good = Q8Case(rows, 2, 2, 64)
    for breakage in ("page", "negative page", "cached", "starts", "max_fresh"):
        case = Q8Case(rows, 2, 2, 64)
        bad, kw = 1, {}
        if breakage == "page":
            case.table[1, 2] = case.q8[0].shape[0]
        elif breakage == "negative page":
            case.table[1, 0] = -3
        elif breakage == "cached":
            case.cached[1] = 16 * case.table.shape[1]
        elif breakage == "starts":
            case.starts[4] = case.P1.shape[0] + 1
            bad = 3
        else:
            kw["max_fresh"] = 45
            bad = 3
        Y, L = case.run(**kw)
        assert rb.relation_check_device_status() == 1, breakage
        lo, hi = int(good.starts[bad]), int(good.starts[bad + 1])
        Q8Case(rows, 2, 2, 64).check(Y, L, only=[n for n in range(good.P1.shape[0]) if not lo <= n < hi])
    good.run()
    assert rb.relation_check_device_status() == 0


@pytest.mark.parametrize("rows", [[(700, 60)], [(700, 1)]])
def test_offsets_past_32_bits(rows):
    """Pages whose byte offsets pass 2^32: the case's pages are the pools' last."""
    page, G, d, pages = 256, 8, 64, 33000
    case = Q8Case(rows, G, G, d, page=page)
    big = rb.paged_pages_q8(pages, G, page, d)
    assert big[0].numel() > 1 << 32
    for b, small in zip(big, case.q8):
        b[-small.shape[0]:] = small.cuda()
    table = torch.where(case.table < (1 << 30), case.table + pages - case.q8[0].shape[0], case.table)
    L = torch.full(case.P1.shape[:2], -7.0, device="cuda")
    Y, _ = rb.paged_fwd_q8(case.P1.cuda(), *big, table.cuda(), case.starts.cuda(), case.cached.cuda(), rows[0][1], case.tau,
                           case.lam, None, L)
    torch.cuda.synchronize()
    assert rb.relation_check_device_status() == 0
    case.check(Y.cpu(), L.cpu(), only=[0, rows[0][1] - 1])


def test_a_step_captured_and_replayed_with_other_lengths():
    """Store and forward in a graph; between replays the lengths, tokens and slots are others."""
    gen = torch.Generator().manual_seed(3)
    H, G, d, page, R, N, width = 4, 2, 64, 16, 3, 40, 8
    pools = rb.paged_pages_q8(R * width, G, page, d)
    table = torch.randperm(R * width, generator=gen).int().view(R, width).cuda()
    X = {k: torch.zeros(N, h, d, dtype=torch.bfloat16, device="cuda") for k, h in (("X1", H), ("X2", G), ("I", G))}
    P1, Y = torch.empty_like(X["X1"]), torch.empty_like(X["X1"])
    starts = torch.zeros(R + 1, dtype=torch.int32, device="cuda")
    cached, positions = torch.zeros(R, dtype=torch.int32, device="cuda"), torch.zeros(N, dtype=torch.int32, device="cuda")
    slots = torch.full((N,), -1, dtype=torch.int64, device="cuda")
    ws = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")

    def step():
        rb.paged_store_q8(X["X1"], X["X2"], X["I"], None, 0, 1e4, positions, slots, P1, *pools)
        rb.paged_fwd_q8(P1, *pools, table, starts, cached, N, 2.0, 0.5, Y, None, ws)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    from oracle import paged as po

    done = [0, 0, 0]
    for fresh in ([20, 1, 19], [1, 30, 0], [3, 2, 1], [1, 1, 1]):
        n, at = sum(fresh), [0]
        for f in fresh:
            at.append(at[-1] + f)
        pos = [c + t for c, f in zip(done, fresh) for t in range(f)]
        of = [r for r, f in enumerate(fresh) for _ in range(f)]
        host = table.cpu()
        sl = [int(host[r, p // page]) * page + p % page for r, p in zip(of, pos)]
        starts.copy_(torch.tensor(at, dtype=torch.int32))
        cached.copy_(torch.tensor(done, dtype=torch.int32))
        positions[:n] = torch.tensor(pos, dtype=torch.int32).cuda()
        slots.fill_(-1)
        slots[:n] = torch.tensor(sl).cuda()
        for x in X.values():
            x[:n] = torch.randn(n, *x.shape[1:], generator=gen).bfloat16().cuda()
        graph.replay()
        torch.cuda.synchronize()
        assert rb.relation_check_device_status() == 0
        held = [(p[..., :d].double() * pools[2][..., k, None].double()).cpu().numpy() for k, p in enumerate(pools[:2])]
        Yr, _ = po.fwd(P1[:n].double().cpu().numpy(), *held, host.numpy(), at, done, 2.0, 0.5, page, 0)
        assert np.abs(Y[:n].double().cpu().numpy() - Yr).max() <= 1e-2 * np.abs(held[1]).max()
        done = [c + f for c, f in zip(done, fresh)]
