"""Continuous batching of a hybrid: Linear Relation layers in front of a Full Relation layer with an 8-bit cache.

A request holds one state of d_h x d_h a head and Linear layer, however long it grows, and pages of the Full layer's
cache at half of bf16's bytes.  A step takes any mix of prompts, chunks and single tokens: linear_packed_fwd for every
Linear layer (linear_step, where each request has one token), then paged_plan, paged_store_q8 and paged_fwd_q8 for the
Full layer; a layer's output is the next one's information states.  The lengths are the host's own, so no step waits
for the GPU.  At the end every request's rows are compared with the dense paths over its whole sequence: the Linear
layers' with relation_linear_fwd_gate, the Full layer's with relation_fwd over the rows that its cache holds.

    python examples/hybrid_serving.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from relation_token_mixing_gb300 import binding as rb  # noqa: E402

TAU_S, LAM, ROPE_BASE, PAIRING = 2.0, 0.5, 1e4, 0


class LinearLayer:
    """One Linear layer's pool of states: request r's is in slot r once it has begun."""

    def __init__(self, requests, heads, d_h, gen):
        self.states = rb.linear_states(requests, heads, d_h)
        self.A_log = torch.log(torch.rand(heads, d_h, generator=gen) + 0.5).cuda()
        self.dt_bias = (torch.randn(heads, d_h, generator=gen) - 3.0).cuda()
        self.workspace = None

    def step(self, P1, P2, I, G, starts, slots_in, slots_out, fresh):
        if all(f == 1 for f in fresh):
            return rb.linear_step(P1, P2, I, G, self.states, slots_in, slots_out, TAU_S, self.A_log, self.dt_bias)
        most = max(fresh)
        prob = rb.linear_packed_for(P1, self.states, len(fresh), TAU_S)
        need = rb.relation_linear_packed_workspace_bytes(prob, most)
        if need and (self.workspace is None or self.workspace.numel() < need):
            self.workspace = torch.empty(need, dtype=torch.uint8, device="cuda")
        return rb.linear_packed_fwd(P1, P2, I, G, starts, self.states, slots_in, slots_out, most, TAU_S, self.A_log,
                                    self.dt_bias, workspace=self.workspace)

    def dense(self, P1, P2, I, G):
        prob = rb.problem_for(P1, TAU_S, 0.0, True, rb.RELATION_LAYOUT_BHTD)
        Y = torch.empty_like(I)
        rb.relation_linear_fwd_gate(prob, P1, P2, I, G, self.A_log, self.dt_bias, Y, None,
                                    rb.linear_workspace(prob, P1.device))
        return Y


class FullLayer:
    """One Full layer's 8-bit pages, the requests' block tables and the free list."""

    def __init__(self, requests, heads, d_h, pages, page_size, width, gen):
        self.page_size, self.pages, self.d_h = page_size, pages, d_h
        self.pools = rb.paged_pages_q8(pages, heads, page_size, d_h)
        self.table = torch.full((requests, width), -1, dtype=torch.int32, device="cuda")
        self.free = torch.randperm(pages, generator=gen).to(torch.int32).cuda()  # any order does
        self.used = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.theta = (torch.randn(heads // 2, generator=gen) * 0.3).cuda()
        self.starts = torch.zeros(requests + 1, dtype=torch.int32, device="cuda")
        self.workspace = None

    def plan(self, lengths, cached, fresh_lengths, fresh):
        """Slots and positions of a step's tokens; starts, which the Linear layers read too."""
        N = sum(fresh_lengths)
        self.slots = torch.empty(N, dtype=torch.int64, device="cuda")
        self.positions = torch.empty(N, dtype=torch.int32, device="cuda")
        rb.paged_plan(cached, fresh, self.free, self.table, self.pages, self.page_size, self.starts, self.slots,
                      self.positions, self.used)
        # What the plan took from the front of the free list, from the lengths alone.
        pages = lambda n: -(-n // self.page_size)  # noqa: E731
        taken = sum(pages(c + f) - pages(c) for c, f in zip(lengths, fresh_lengths))
        self.free = self.free[taken:].contiguous()

    def step(self, X1, X2, I, cached, fresh):
        P1, most = torch.empty_like(X1), max(fresh)
        rb.paged_store_q8(X1, X2, I, self.theta, PAIRING, ROPE_BASE, self.positions, self.slots, P1, *self.pools)
        prob = rb.paged_q8_for(*X1.shape, *self.pools, len(fresh), self.table.shape[1], TAU_S, LAM,
                               rb.RELATION_LAYOUT_BHTD)
        need = rb.relation_paged_q8_workspace_bytes(prob, most)
        if self.workspace is None or self.workspace.numel() < need:
            self.workspace = torch.empty(need, dtype=torch.uint8, device="cuda")
        Y, _ = rb.paged_fwd_q8(P1, *self.pools, self.table, self.starts, cached, most, TAU_S, LAM,
                               workspace=self.workspace)
        return Y

    def dense(self, r, X1):
        """Request r's rows by the dense path: X1 [1, H, T, d_h] against the rows that the cache holds."""
        T = X1.shape[2]
        j = torch.arange(T, device="cuda")
        slots = self.table[r].long()[j // self.page_size] * self.page_size + j % self.page_size
        P2, I = (x.transpose(0, 1).unsqueeze(0).contiguous() for x in rb.paged_read_q8(slots, *self.pools, self.d_h))
        P1, *unused = (torch.empty_like(X1) for _ in range(3))
        rb.relation_prologue_fwd(rb.problem_for(X1, TAU_S, LAM, True), X1, X1, X1, self.theta, PAIRING, ROPE_BASE, None,
                                 P1, *unused)
        return rb.fwd(P1, P2, I, TAU_S, LAM, True)[0], float(I.float().abs().max())


def main(prompts=(700, 33, 1, 256, 90), decode=6, chunk=256, heads=8, d_h=60, page_size=64, linear_layers=3):
    """Serves the prompts; returns the largest differences to the dense paths, of any Linear layer relative to max |Y|
    and of the Full layer relative to max |I~|."""
    gen = torch.Generator().manual_seed(5)
    total = [p + decode for p in prompts]
    rand = lambda t, shift=0.0: torch.randn(t, heads, d_h, generator=gen) + shift  # noqa: E731
    # Every layer's relation coordinates (a model's projections), the retention's inputs and the first states.
    X = [[[rand(t).bfloat16().cuda() for t in total] for _ in range(2)] for _ in range(linear_layers + 1)]
    R = [[rand(t).cuda() for t in total] for _ in range(linear_layers)]
    I0 = [rand(t).bfloat16().cuda() for t in total]
    linear = [LinearLayer(len(prompts), heads, d_h, gen) for _ in range(linear_layers)]
    pages = sum(-(-t // page_size) for t in total) + 3
    full = FullLayer(len(prompts), heads, d_h, pages, page_size, -(-max(total) // page_size), gen)
    lengths = [0] * len(prompts)
    outputs = [[[] for _ in prompts] for _ in range(linear_layers + 1)]
    steps = 0
    while any(n < t for n, t in zip(lengths, total)):
        # A prompt's next chunk, or one token; requests arrive one step after another.
        fresh = [0 if steps < r else min(chunk, p - n) if n < p else min(1, t - n)
                 for r, (n, p, t) in enumerate(zip(lengths, prompts, total))]
        ints = lambda x: torch.tensor(x, dtype=torch.int32).pin_memory().cuda(non_blocking=True)  # noqa: E731
        new = lambda xs: torch.cat([x[n: n + f] for x, n, f in zip(xs, lengths, fresh)])  # noqa: E731
        cached = ints(lengths)
        full.plan(lengths, cached, fresh, ints(fresh))
        slots_in = ints([r if n else -1 for r, n in enumerate(lengths)])  # a new request has no state yet
        slots_out = ints([r if n + f else -1 for r, (n, f) in enumerate(zip(lengths, fresh))])
        Y = new(I0)
        for k, layer in enumerate(linear):
            Y = layer.step(new(X[k][0]), new(X[k][1]), Y, new(R[k]), full.starts, slots_in, slots_out, fresh)
            for out, part in zip(outputs[k], Y.split(fresh)):
                out.append(part)
        Y = full.step(new(X[-1][0]), new(X[-1][1]), Y, cached, fresh)
        for out, part in zip(outputs[-1], Y.split(fresh)):
            out.append(part)
        lengths = [n + f for n, f in zip(lengths, fresh)]
        steps += 1
    torch.cuda.synchronize()
    if rb.relation_check_device_status() != 0:
        raise RuntimeError("a device-side wait expired or an index was out of range")
    worst_linear = worst_full = 0.0
    rows = lambda x: x.transpose(0, 1).unsqueeze(0).contiguous()  # noqa: E731  [1, heads, T, d_h]
    for r in range(len(prompts)):
        got = [rows(torch.cat(out[r])) for out in outputs]
        for k, layer in enumerate(linear):  # each layer from the served states of the one before
            want = layer.dense(rows(X[k][0][r]), rows(X[k][1][r]), got[k - 1] if k else rows(I0[r]), rows(R[k][r]))
            diff = (got[k].float() - want.float()).abs().max() / want.float().abs().max()
            worst_linear = max(worst_linear, float(diff))
        want, largest = full.dense(r, rows(X[-1][0][r]))
        worst_full = max(worst_full, float((got[-1].float() - want.float()).abs().max()) / largest)
    print(f"{len(prompts)} requests, {sum(total)} tokens in {steps} steps: largest difference to the dense paths, Linear "
          f"{worst_linear:.1e} of max |Y|, Full {worst_full:.1e} of max |I~|")
    return worst_linear, worst_full


if __name__ == "__main__":
    if max(main()) > 2e-2:  # both sides are within 1e-2 of the formulas
        sys.exit(1)
