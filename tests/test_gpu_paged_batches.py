"""The paged forward as a server uses it: batches of more requests than a block has threads (the schedule's sums take
several rounds), calls one after another over one workspace, and a captured step replayed with other lengths."""
import numpy as np
import pytest
import torch

from relation_token_mixing_gb300 import binding as rb
from test_gpu_paged import BF, BTHD, F32, Case

pytestmark = pytest.mark.gpu


def _rows(R, seed, few, long=0, cached=60):
    """R requests, two thirds of them without new tokens, `long` of them with 40 to 90."""
    r = np.random.default_rng(seed)
    rows = [(int(r.integers(0, cached)), int(r.integers(1, few + 1)) if r.random() < 1 / 3 else 0) for _ in range(R)]
    for k in r.choice(R, long, replace=False):
        rows[k] = (int(r.integers(0, cached)), int(r.integers(40, 91)))
    rows[-1] = (cached, 1)
    return rows


BATCHES = {
    "decode_d64": dict(H=4, G=2, d=64, page=16), "few_d128": dict(H=4, G=2, d=128, page=32, layout=BTHD),
    "long_d64": dict(H=2, G=2, d=64, page=16, layout=BTHD), "long_d80": dict(H=4, G=2, d=80, page=64),
    "f32_d64": dict(H=2, G=1, d=64, page=16, dtype=F32), "f32_long_d128": dict(H=2, G=2, d=128, page=16, dtype=F32)}


@pytest.mark.parametrize("R", [400, 1025, 8192])
@pytest.mark.parametrize("name", list(BATCHES))
def test_forward_of_more_requests_than_threads(name, R):
    rows = _rows(R, R, 3 if "few" in name else 1, R // 50 if "long" in name else 0)
    case = Case(rows, **BATCHES[name], extra=2)
    Y, L = case.run()
    assert rb.relation_check_device_status() == 0
    ends = [n for n, (_, f) in zip(case.starts[1:].tolist(), rows) if f]
    rng = np.random.default_rng(0)
    sample = sorted({0, ends[-1] - 1, *(ends[k] - 1 for k in rng.integers(0, len(ends), 60))})
    assert torch.isfinite(Y[: ends[-1]].float()).all() and not (L[: ends[-1]] == -7.0).any()
    case.check(Y, L, only=sample)


@pytest.mark.parametrize("dtype,d", [(BF, 64), (BF, 128), (F32, 64)])
def test_calls_one_after_another_over_one_workspace(dtype, d):
    """Eight calls in flight at once, of different batches, over one workspace and one Y each, give what each gives
    alone."""
    shapes = [[(3000, 1), (7, 1)], [(0, 300), (900, 40)], [(5000, 2), (100, 90), (0, 1)], [(64, 200)]]
    cases = [Case(shapes[k % 4], 4, 2, d, page=32, dtype=dtype, seed=k) for k in range(8)]
    args, most, sizes = [], [], []
    for c in cases:
        dev = [x.cuda() for x in (c.P1, *c.pools, c.table, c.starts, c.cached)]
        args.append(dev)
        most.append(max(f for _, f in c.rows))
        prob = rb.paged_for(dev[0], dev[1], len(c.rows), c.table.shape[1], c.tau, c.lam, c.layout)
        sizes.append(rb.relation_paged_workspace_bytes(prob, most[-1]))
    alone = []
    for c, dev, m in zip(cases, args, most):
        alone.append(rb.paged_fwd(*dev, m, c.tau, c.lam)[0])
        torch.cuda.synchronize()
    ws = torch.full((max(sizes) // 4,), float("nan"), device="cuda")
    for _ in range(5):
        out = [torch.full_like(dev[0], -7.0) for dev in args]
        torch.cuda.synchronize()
        for c, dev, m, Y in zip(cases, args, most, out):
            rb.paged_fwd(*dev, m, c.tau, c.lam, Y, None, ws)
        torch.cuda.synchronize()
        assert rb.relation_check_device_status() == 0
        for a, b in zip(alone, out):
            assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_a_captured_step_replayed_with_other_lengths(dtype):
    """plan, store and forward in a graph, captured once; each replay has other lengths, tokens and free pages in the
    same buffers (N and max_fresh are bounds, so a step may have fewer new tokens) and gives what the calls give."""
    R, H, G, d, page, width, pages, N, bound = 5, 4, 2, 64, 16, 40, 160, 120, 100
    g = torch.Generator().manual_seed(3)
    steps = [([0, 0, 0, 0, 0], [100, 1, 0, 10, 9]), ([100, 1, 0, 10, 9], [1, 1, 1, 1, 1]),
             ([101, 2, 1, 11, 10], [0, 3, 60, 0, 57]), ([101, 5, 61, 11, 67], [1, 0, 1, 0, 1])]
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731

    class Step:
        def __init__(self):
            self.cached, self.fresh, self.free = i32(R), i32(R), i32(pages)
            self.table, self.starts, self.pos, self.used = i32(R, width) - 1, i32(R + 1), i32(N), i32(1)
            self.slots = torch.zeros(N, dtype=torch.int64, device="cuda")
            self.X1, self.X2, self.I = (torch.zeros(N, h, d, dtype=dtype, device="cuda") for h in (H, G, G))
            self.theta = torch.full((G // 2,), 0.3, device="cuda")
            self.pools = rb.paged_pages(pages, G, page, d, dtype)
            self.P1, self.Y = torch.zeros_like(self.X1), torch.zeros_like(self.X1)
            prob = rb.paged_for(self.P1, self.pools[0], R, width, 1.0, 0.5, rb.RELATION_LAYOUT_BHTD)
            self.ws = rb.paged_workspace(prob, bound)

        def fill(self, cached, fresh, free, xs):
            for t, v in ((self.cached, cached), (self.fresh, fresh), (self.free, free)):
                t.copy_(torch.as_tensor(v, dtype=torch.int32))
            for t, v in zip((self.X1, self.X2, self.I), xs):
                t.copy_(v)
            self.Y.fill_(-7.0)

        def run(self):
            rb.paged_plan(self.cached, self.fresh, self.free, self.table, pages, page, self.starts, self.slots, self.pos,
                          self.used)
            rb.paged_store(self.X1, self.X2, self.I, self.theta, 0, 1e4, self.pos, self.slots, self.P1, *self.pools)
            rb.paged_fwd(self.P1, *self.pools, self.table, self.starts, self.cached, bound, 1.0, 0.5, self.Y, None, self.ws)

    plain, captured = Step(), Step()
    captured.run()  # an empty step, before the capture
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured.run()
    order, taken = torch.randperm(pages, generator=g), 0
    for cached, fresh in steps:
        xs = [torch.randn(N, h, d, generator=g).to(dtype) for h in (H, G, G)]
        free = torch.cat([order[taken:], order[:taken]])
        for s in (plain, captured):
            s.fill(cached, fresh, free, xs)
        plain.run()
        graph.replay()
        torch.cuda.synchronize()
        assert rb.relation_check_device_status() == 0
        for a, b in zip((plain.table, plain.starts, plain.slots, plain.pos, plain.used, plain.P1, *plain.pools, plain.Y),
                        (captured.table, captured.starts, captured.slots, captured.pos, captured.used, captured.P1,
                         *captured.pools, captured.Y)):
            assert torch.equal(a, b)
        n = sum(fresh)
        assert (captured.Y[:n] != -7.0).any(-1).all() and (captured.Y[n:] == -7.0).all()
        taken += int(plain.used)
