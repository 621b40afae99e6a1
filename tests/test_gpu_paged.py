"""GPU parity of the paged Relation Cache ("Ask Self, Ask Others", Sec. 5.3 eq.(18), Appendix A.5) through the C ABI,
against the float64 oracle.

Every slot that holds no token of the case is NaN (unused pages, the ends of last pages, the rows of page padding),
block-table entries past a request's pages are far out of range, workspaces start as NaN, and Y, L rows outside the
requests keep a sentinel: reading or writing one of them shows.
Tolerances, as for the operator itself: Y <= 1e-5 max|V| (fp32), 1e-2 max|V| (bf16); L <= 1e-6 max(1, |L|) plus
len 2^-24 (fp32), 1e-3 max(1, |L|) (bf16).  Stored rows: 2e-6 max|x| (fp32: two products of values rounded to 2^-24,
and an angle within 4e-7), 2^-8 max|x| (bf16: one rounding of a value of at most sqrt(2) max|x|, 2^-9 sqrt(2), and the
fp32 part).  Whole numbers are equal.
"""
import numpy as np
import pytest
import torch

from oracle import paged as po
from relation_token_mixing_gb300 import binding as rb

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
BHTD, BTHD = rb.RELATION_LAYOUT_BHTD, rb.RELATION_LAYOUT_BTHD
SENTINEL = -7.0


def _status_ok():
    torch.cuda.synchronize()
    assert rb.relation_check_device_status() == 0


# ---------------------------------------------------------------------- plan
PLANS = [
    # cached, fresh, page, free list longer (+) or shorter (-) than needed, extra rows in the packed tensors
    ([0], [1], 16, 0, 0),
    ([5], [0], 16, 3, 4),
    ([9, 3, 16, 0], [8, 0, 1, 17], 16, 2, 0),
    ([9, 3, 16, 0], [8, 0, 1, 17], 16, -1, 3),
    ([31, 32, 33, 0, 255], [1, 1, 1, 1, 1], 32, 0, 0),
    ([0] * 7, [0, 0, 3000, 0, 1, 0, 0], 64, 5, 100),
    (list(range(0, 2500)), [k % 4 for k in range(2500)], 16, 10, 1),
    ([1000 - k % 300 for k in range(1500)], [1] * 1500, 256, 0, 0),
]


@pytest.mark.parametrize("cached,fresh,page,spare,extra", PLANS)
def test_plan(cached, fresh, page, spare, extra):
    rng = np.random.default_rng(len(cached) + page)
    R, N = len(cached), sum(fresh) + extra
    held = [-(-c // page) for c in cached]
    new = sum(-(-(c + f) // page) - h for c, f, h in zip(cached, fresh, held))
    pages = sum(held) + max(0, new + spare) + 1
    ids = rng.permutation(pages)
    width = max(-(-(c + f) // page) for c, f in zip(cached, fresh)) + 1
    table = np.full((R, width), -1)
    at = 0
    for r in range(R):
        table[r, : held[r]] = ids[at: at + held[r]]
        at += held[r]
    free = ids[at: at + max(0, new + spare)]
    want = po.plan(cached, fresh, free, table, pages, page, N)
    dev = lambda x, dt=torch.int32: torch.tensor(np.asarray(x), dtype=dt, device="cuda")  # noqa: E731
    t, starts = dev(table), torch.full((R + 1,), 99, dtype=torch.int32, device="cuda")
    slots, pos = dev(np.full(N, 99), torch.int64), dev(np.full(N, 99))
    used = torch.full((1,), 99, dtype=torch.int32, device="cuda")
    for _ in range(2):  # the second pass finds its own entries in the table
        rb.paged_plan(dev(cached), dev(fresh), dev(free) if len(free) else None, t, pages, page, starts, slots, pos, used)
        _status_ok()
        for got, ref in zip((t, starts, slots, pos, used), want):
            np.testing.assert_array_equal(got.cpu().numpy().reshape(-1), np.asarray(ref).reshape(-1))


def test_plan_past_the_table_and_bad_entries():
    """Tokens past the table's width and tokens of pages outside the pool get slot -1, and no page."""
    dev = lambda x, dt=torch.int32: torch.tensor(x, dtype=dt, device="cuda")  # noqa: E731
    cached, fresh, table, free = [30, 20, 5], [10, 3, 2], [[1, 0], [0, 900], [-5, -1]], [3, 2]
    want = po.plan(cached, fresh, free, table, 4, 16, 15)
    t, starts, slots, pos, used = dev(table), dev([0] * 4), dev([0] * 15, torch.int64), dev([0] * 15), dev([0])
    rb.paged_plan(dev(cached), dev(fresh), dev(free), t, 4, 16, starts, slots, pos, used)
    _status_ok()
    for got, ref in zip((t, starts, slots, pos, used), want):
        np.testing.assert_array_equal(got.cpu().numpy().reshape(-1), np.asarray(ref).reshape(-1))


def test_plan_reports_bad_lengths():
    dev = lambda x, dt=torch.int32: torch.tensor(x, dtype=dt, device="cuda")  # noqa: E731
    for cached, fresh, N in (([3, -1], [1, 1], 4), ([3, 1], [1, -9], 4), ([0, 0], [3, 3], 4)):
        t, starts, slots, pos, used = dev([[0], [1]]), dev([0] * 3), dev([0] * N, torch.int64), dev([0] * N), dev([0])
        rb.paged_plan(dev(cached), dev(fresh), None, t, 4, 16, starts, slots, pos, used)
        torch.cuda.synchronize()
        assert rb.relation_check_device_status() == 1


# --------------------------------------------------------------------- store
def _pools(pages, G, page, d, dtype, layout, fill=float("nan")):
    return [p.fill_(fill) for p in rb.paged_pages(pages, G, page, d, dtype, layout)]


STORES = [
    (1, 1, 1, 64, 16, BF, BHTD, None), (7, 8, 8, 64, 16, BF, BTHD, 0), (33, 8, 2, 128, 64, BF, BHTD, 1),
    (50, 4, 4, 60, 32, BF, BHTD, 0), (50, 4, 4, 60, 32, BF, BTHD, 1), (21, 6, 2, 48, 256, BF, BTHD, 0),
    (1300, 10, 10, 80, 16, BF, BHTD, 1), (9, 4, 2, 60, 16, F32, BHTD, 0), (700, 3, 3, 64, 128, F32, BTHD, None),
    (5000, 4, 4, 48, 64, F32, BHTD, 1), (77, 2, 2, 80, 16, F32, BTHD, 0), (40, 4, 2, 128, 32, F32, BHTD, 0)]


@pytest.mark.parametrize("N,H,G,d,page,dtype,layout,pairing", STORES)
@pytest.mark.parametrize("base", [1e4, 0.0])
def test_store(N, H, G, d, page, dtype, layout, pairing, base):
    g = torch.Generator().manual_seed(N + d)
    X1, X2, I = (torch.randn(N, h, d, generator=g).to(dtype) for h in (H, G, G))
    theta = None if pairing is None else torch.randn(G // 2, generator=g)
    positions = torch.randint(0, 40000, (N,), generator=g).int()
    pages = -(-N // page) + 2
    slots = torch.randperm(pages * page, generator=g)[:N]
    slots[N // 2] = -1
    pools = _pools(pages, G, page, d, dtype, layout)
    P1 = torch.empty_like(X1, device="cuda")
    rb.paged_store(X1.cuda(), X2.cuda(), I.cuda(), None if theta is None else theta.cuda(), pairing or 0, base,
                   positions.cuda(), slots.cuda(), P1, *pools, layout)
    _status_ok()
    nan = [np.full(p.shape, np.nan) for p in pools]
    ref = po.store(X1.double(), X2.double(), I.double(), None if theta is None else theta.double().numpy(),
                   pairing or 0, base, positions.numpy(), slots.numpy(), *nan, page, layout)
    for got, want, x in zip((P1, *pools), ref, (X1, X2, I)):
        got, tol = got.double().cpu().numpy(), (2e-6 if dtype is F32 else 2.0 ** -8) * float(x.double().abs().max())
        if got.shape[-1] != d and got.ndim == 4:  # the padding of 60-wide rows is nobody's
            got, want = got[..., :d], want[..., :d]
        np.testing.assert_array_equal(np.isnan(got), np.isnan(want))
        assert np.nanmax(np.abs(got - want), initial=0.0) <= tol


def test_store_reports_a_slot_past_the_pool():
    X = torch.ones(2, 2, 64, dtype=BF, device="cuda")
    pools = _pools(2, 2, 16, 64, BF, BHTD)
    P1 = torch.empty_like(X)
    rb.paged_store(X, X, X, None, 0, 1e4, torch.zeros(2, dtype=torch.int32, device="cuda"),
                   torch.tensor([3, 32], device="cuda"), P1, *pools)
    torch.cuda.synchronize()
    assert rb.relation_check_device_status() == 1
    assert int(torch.isfinite(pools[0]).sum()) == 2 * 64 and torch.equal(P1, X)


# ------------------------------------------------------------------- forward
class Case:
    """A paged cache of random tokens: pages in random order, everything unused NaN."""

    def __init__(self, rows, H, G, d, page=16, dtype=BF, layout=BHTD, tau=1.0, lam=0.5, scale=1.0, seed=0, extra=0,
                 first=0):
        self.rows, self.page, self.layout, self.tau, self.lam, self.d = rows, page, layout, tau, lam, d
        g = torch.Generator().manual_seed(seed)
        rng = np.random.default_rng(seed)
        need = [-(-(c + f) // page) for c, f in rows]
        pages, width = sum(need) + 3, max(max(need), 1)
        ids, at = rng.permutation(pages), 0
        table = np.full((len(rows), width), 1 << 30)
        self.pools = [p.cpu() for p in _pools(pages, G, page, d, dtype, layout)]
        for r, k in enumerate(need):
            table[r, :k] = ids[at: at + k]
            at += k
        pos = np.concatenate([np.arange(c + f) for c, f in rows] + [np.zeros(0, dtype=int)])
        req = np.concatenate([np.full(c + f, r) for r, (c, f) in enumerate(rows)] + [np.zeros(0, dtype=int)])
        pid, off = torch.from_numpy(table[req, pos // page]), torch.from_numpy(pos % page)
        for pool, sc in zip(self.pools, (scale, 1.0)):
            x = (torch.randn(len(pos), G, d, generator=g) * sc).to(dtype)
            view = pool if layout == BTHD else pool.transpose(1, 2)
            view[pid, off, :, :d] = x
        fresh = [f for _, f in rows]
        N = first + sum(fresh) + extra
        self.P1 = (torch.randn(N, H, d, generator=g) * scale).to(dtype)
        self.starts = torch.tensor(first + np.concatenate([[0], np.cumsum(fresh)]), dtype=torch.int32)
        self.cached = torch.tensor([c for c, _ in rows], dtype=torch.int32)
        self.table = torch.tensor(table, dtype=torch.int32)
        self.vmax = float(torch.nan_to_num(self.pools[1].double()).abs().max())

    def run(self, max_fresh=None, stream=None):
        dev = [x.cuda() for x in (self.P1, *self.pools, self.table, self.starts, self.cached)]
        Y = torch.full_like(dev[0], SENTINEL)
        L = torch.full(self.P1.shape[:2], SENTINEL, device="cuda")
        m = max(f for _, f in self.rows) if max_fresh is None else max_fresh
        prob = rb.paged_for(dev[0], dev[1], len(self.rows), self.table.shape[1], self.tau, self.lam, self.layout)
        ws = torch.full((rb.relation_paged_workspace_bytes(prob, m) // 4 + 4,), float("nan"), device="cuda")
        torch.cuda.synchronize()
        rb.paged_fwd(*dev, m, self.tau, self.lam, Y, L, ws, self.layout, stream)
        torch.cuda.synchronize()
        return Y.cpu(), L.cpu()

    def check(self, Y, L, only=None):
        ref, refL = po.fwd(self.P1.double(), *(p.double().numpy() for p in self.pools), self.table.numpy(),
                           self.starts.numpy(), self.cached.numpy(), self.tau, self.lam, self.page, self.layout, only)
        got, gotL = Y.double().numpy(), L.double().numpy()
        lo, hi = int(self.starts[0]), int(self.starts[-1])
        assert (got[:lo] == SENTINEL).all() and (got[hi:] == SENTINEL).all()
        assert (gotL[:lo] == SENTINEL).all() and (gotL[hi:] == SENTINEL).all()
        rows = ~np.isnan(refL).any(1)
        f32 = self.P1.dtype is F32
        err = np.abs(got[rows] - ref[rows]).max(initial=0.0)
        assert err <= (1e-5 if f32 else 1e-2) * self.vmax, err
        longest = max(c + f for c, f in self.rows)
        tolL = (1e-6 if f32 else 1e-3) * np.maximum(1.0, np.abs(refL[rows])) + (longest * 2.0 ** -24 if f32 else 0.0)
        assert (np.abs(gotL[rows] - refL[rows]) <= tolL).all(), np.abs(gotL[rows] - refL[rows]).max()


EDGES = [(0, 1), (1, 1), (15, 1), (16, 1), (17, 1), (31, 2), (32, 1), (33, 3), (63, 1), (64, 4), (127, 1), (128, 1),
         (129, 2), (0, 5), (40, 0), (255, 1), (0, 0), (256, 1), (300, 3)]
FWD = {
    "decode_edges_d64": dict(rows=EDGES, H=4, G=4, d=64),
    "decode_edges_g2_d64": dict(rows=EDGES, H=4, G=2, d=64, page=32, layout=BTHD),
    "decode_edges_g4_d128": dict(rows=EDGES, H=8, G=2, d=128, page=64),
    "decode_edges_g3_d80": dict(rows=EDGES, H=6, G=2, d=80, page=128, layout=BTHD),
    "decode_edges_d48": dict(rows=EDGES, H=2, G=2, d=48, page=256),
    "decode_edges_g5_d60": dict(rows=EDGES, H=5, G=1, d=60, page=16),
    "decode_edges_g17_d64": dict(rows=EDGES[:9], H=17, G=1, d=64, page=16),
    "decode_long": dict(rows=[(9000, 1), (12, 1), (4097, 1)], H=4, G=2, d=64, page=64),
    "decode_one_long_d128": dict(rows=[(20011, 1)], H=4, G=1, d=128, page=16),
    "decode_many": dict(rows=[(k * 7 % 97, 1) for k in range(300)], H=2, G=1, d=64, page=16),
    "few_rows": dict(rows=[(500 + k, 1 + k % 9) for k in range(12)], H=8, G=2, d=64, page=32),
    "few_rows_d128": dict(rows=[(300 + 50 * k, 1 + k % 5) for k in range(9)], H=8, G=2, d=128, page=16, layout=BTHD),
    "prompts_d64": dict(rows=[(0, 1), (0, 300), (0, 129), (0, 0), (0, 64), (0, 513)], H=2, G=2, d=64, page=64),
    "prompts_g4_d128": dict(rows=[(0, 100), (0, 257), (0, 31)], H=4, G=1, d=128, page=32),
    "chunk_d64": dict(rows=[(1000, 200), (37, 300), (511, 70)], H=2, G=2, d=64, page=16, layout=BTHD),
    "chunk_g3_d80": dict(rows=[(700, 150), (5, 90)], H=6, G=2, d=80, page=128),
    "chunk_g2_d60": dict(rows=[(700, 150), (5, 90)], H=4, G=2, d=60, page=32),
    "chunk_g7_d48": dict(rows=[(300, 61), (1, 40)], H=7, G=1, d=48, page=16),
    "chunk_long_d128": dict(rows=[(6000, 140)], H=2, G=1, d=128, page=64),
    "chunk_long_few_rows_d64": dict(rows=[(9000, 40)], H=1, G=1, d=64, page=256, layout=BTHD),
    "mixed": dict(rows=[(900, 1), (0, 200), (33, 0), (2000, 1), (64, 64), (7, 3)], H=4, G=2, d=64, page=16),
    "mixed_d128": dict(rows=[(900, 1), (0, 200), (33, 0), (2000, 1), (64, 64), (7, 3)], H=4, G=2, d=128, page=32),
    "big_evidence": dict(rows=[(600, 3), (100, 90), (0, 200)], H=2, G=2, d=64, tau=0.5, scale=6.0),
    "no_correction": dict(rows=[(600, 1), (100, 90)], H=2, G=1, d=64, lam=0.0),
    "negative_correction_d128": dict(rows=[(600, 1), (100, 90)], H=2, G=1, d=128, lam=-0.75, tau=0.7),
    "f32_d64": dict(rows=[(0, 1), (70, 1), (33, 40), (0, 90), (64, 0), (500, 3)], H=4, G=2, d=64, dtype=F32),
    "f32_d128": dict(rows=[(300, 1), (33, 70), (0, 65)], H=2, G=2, d=128, dtype=F32, page=64, layout=BTHD),
    "f32_d60": dict(rows=[(300, 1), (33, 70), (0, 65)], H=3, G=1, d=60, dtype=F32, page=32),
    "f32_d48": dict(rows=[(15, 1), (16, 20), (1, 1)], H=2, G=2, d=48, dtype=F32, page=16, layout=BTHD),
    "f32_d80_long": dict(rows=[(5000, 2), (100, 130)], H=2, G=1, d=80, dtype=F32, page=128),
}


@pytest.mark.parametrize("name", list(FWD))
def test_forward(name):
    case = Case(**FWD[name], extra=3)
    Y, L = case.run()
    assert rb.relation_check_device_status() == 0
    case.check(Y, L)


LONG = {  # so many heads that a block's pieces are many tiles long, ends inside tiles among them
    "long_pieces_d64": dict(rows=[(0, 2000), (77, 300)], H=32, G=32, d=64, page=64),
    "long_pieces_g4_d128": dict(rows=[(3001, 700), (0, 1100)], H=64, G=16, d=128, page=32, layout=BTHD),
    "long_pieces_d80": dict(rows=[(1, 1999)], H=40, G=40, d=80, page=128),
    "long_histories_d64": dict(rows=[(4000, 1), (9000, 3), (300, 1), (5000, 2)], H=32, G=16, d=64, page=16),
    "long_f32_d64": dict(rows=[(500, 700), (0, 333)], H=24, G=24, d=64, page=16, dtype=F32),
}


@pytest.mark.parametrize("name", list(LONG))
def test_forward_over_long_pieces(name):
    case = Case(**LONG[name], extra=1)
    Y, L = case.run()
    assert rb.relation_check_device_status() == 0
    assert torch.isfinite(Y[: int(case.starts[-1])].float()).all()
    rng = np.random.default_rng(1)
    ends = case.starts[1:].tolist()
    case.check(Y, L, only=sorted({*rng.integers(0, ends[-1], 12).tolist(), 0, *(e - 1 for e in ends)}))


@pytest.mark.parametrize("name", ["mixed", "mixed_d128", "few_rows", "f32_d64", "decode_long", "chunk_d64"])
def test_forward_is_the_same_from_run_to_run(name):
    case = Case(**FWD[name])
    (Y, L), (Y2, L2) = case.run(), case.run()
    assert torch.equal(Y, Y2) and torch.equal(L, L2)


@pytest.mark.parametrize("name", ["mixed", "decode_edges_d64", "f32_d64"])
def test_forward_without_a_known_bound_on_a_stream_of_its_own(name):
    """max_fresh = 0 (none known), packed rows that begin after others', a side stream."""
    case = Case(**FWD[name], first=5, extra=2)
    Y, L = case.run(max_fresh=0, stream=torch.cuda.Stream())
    assert rb.relation_check_device_status() == 0
    case.check(Y, L)


def test_forward_offsets_past_32_bits():
    """Pages whose element offsets pass 2^31: the pools hold 2.2e9 elements and the case's pages are their last."""
    page, G, d, c, f = 256, 8, 128, 700, 60
    pages = 8400
    pools = [torch.empty(pages, G, page, d, dtype=BF, device="cuda") for _ in range(2)]
    for rows in ([(c, f)], [(c, 1)]):
        case = Case(rows, G, G, d, page=page)
        for big, small in zip(pools, case.pools):
            big[-small.shape[0]:] = small.cuda()
        table = torch.where(case.table < (1 << 30), case.table + pages - case.pools[0].shape[0], case.table)
        L = torch.full(case.P1.shape[:2], SENTINEL, device="cuda")
        Y, _ = rb.paged_fwd(case.P1.cuda(), *pools, table.cuda(), case.starts.cuda(), case.cached.cuda(), rows[0][1],
                            case.tau, case.lam, None, L)
        _status_ok()
        case.check(Y.cpu(), L.cpu(), only=[0, rows[0][1] - 1])


@pytest.mark.parametrize("dtype", [BF, F32])
def test_forward_skips_and_reports_what_it_cannot_follow(dtype):
    """A page outside the pool reads as zeros, a request longer than its table or than max_fresh is skipped; all are
    reported, and the other requests' rows stay right."""
    rows = [(100, 1), (50, 40), (20, 2), (300, 60)]
    good = Case(rows, 2, 2, 64, dtype=dtype)
    for breakage in ("page", "negative page", "cached", "starts", "max_fresh"):
        case = Case(rows, 2, 2, 64, dtype=dtype)
        bad, kw = 1, {}
        if breakage == "page":
            case.table[1, 2] = case.pools[0].shape[0]
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
        ref = Case(rows, 2, 2, 64, dtype=dtype)
        keep = [n for n in range(good.P1.shape[0]) if not lo <= n < hi]
        ref.check(Y, L, only=keep)
    Y, L = good.run()
    assert rb.relation_check_device_status() == 0


def test_a_step_from_lengths_to_output():
    """plan, store and forward together: two chunks of a prompt and then single tokens give the rows that the causal
    operator gives over the whole prompt."""
    from relation_token_mixing_gb300 import inputs as rin

    B, H, T, d, page = 2, 4, 150, 64, 16
    x = rin.make(rin.Workload("paged", B, H, T, d, BF, 2.0, 0.5, True))
    Yr, _ = rb.fwd(x["P1"].cuda(), x["P2"].cuda(), x["V"].cuda(), 2.0, 0.5)
    pools = rb.paged_pages(24, H, page, d, BF)
    table = torch.full((B, 10), -1, dtype=torch.int32, device="cuda")
    free = torch.randperm(24, device="cuda").int()
    done, taken = [0] * B, 0
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    for step in ([100, 64], [40, 80], [1, 1], [1, 1], [1, 0], [1, 2]):
        N = sum(step)
        starts, pos, used = ints([0] * (B + 1)), ints([0] * N), ints([0])
        slots = torch.empty(N, dtype=torch.int64, device="cuda")
        rb.paged_plan(ints(done), ints(step), free[taken:], table, 24, page, starts, slots, pos, used)
        rows = lambda k: torch.cat([x[k][b, :, done[b]: done[b] + n].transpose(0, 1) for b, n in enumerate(step)]).cuda()  # noqa: E731,B023
        P1 = torch.empty(N, H, d, dtype=BF, device="cuda")
        rb.paged_store(rows("P1"), rows("P2"), rows("V"), None, 0, 0.0, pos, slots, P1, *pools)
        Y, _ = rb.paged_fwd(P1, *pools, table, starts, ints(done), max(step), 2.0, 0.5)
        _status_ok()
        want = torch.cat([Yr[b, :, done[b]: done[b] + n].transpose(0, 1) for b, n in enumerate(step)])
        # both sides are within 1e-2 max|V| of the exact rows
        assert float((Y.float() - want.float()).abs().max()) <= 2e-2 * float(x["V"].float().abs().max())
        taken += int(used)
        done = [c + n for c, n in zip(done, step)]
