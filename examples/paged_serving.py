"""Continuous batching over a paged Relation Cache.

Requests of different lengths arrive, are read in as prompts (the long ones in chunks) and then decode a few tokens
each, all in mixed steps.  A step is three calls: paged_plan (block tables, slots and positions from the lengths),
paged_store (RoPE, Givens mixing and the scatter into pages) and paged_fwd (Relation of the new tokens over the pages).
The lengths are the host's own, so no step waits for the GPU.  At the end every request's rows are compared with the
dense path over its whole sequence.

    python examples/paged_serving.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from relation_token_mixing_gb300 import binding as rb  # noqa: E402

TAU_S, LAM, ROPE_BASE, PAIRING = 2.0, 0.5, 1e4, 0


class PagedCache:
    """One layer's pages, the requests' block tables and the free list."""

    def __init__(self, requests, heads, d_h, pages, page_size, width, dtype=torch.bfloat16, device="cuda"):
        self.page_size, self.pages, self.device = page_size, pages, device
        self.P2, self.I = rb.paged_pages(pages, heads, page_size, d_h, dtype, device=device)
        self.table = torch.full((requests, width), -1, dtype=torch.int32, device=device)
        self.free = torch.randperm(pages).to(torch.int32).to(device)  # any order does
        self.lengths = [0] * requests
        self.used = torch.zeros(1, dtype=torch.int32, device=device)
        self.workspace = None

    def step(self, X1, X2, I, theta, fresh):
        """Relation of fresh[r] new tokens of each request r, packed one request after another: [N, heads, d_h]."""
        N, most = X1.shape[0], max(fresh)
        ints = lambda x: torch.tensor(x, dtype=torch.int32).pin_memory().to(self.device, non_blocking=True)  # noqa: E731
        cached, starts = ints(self.lengths), ints([0] * (len(fresh) + 1))
        slots = torch.empty(N, dtype=torch.int64, device=self.device)
        positions = torch.empty(N, dtype=torch.int32, device=self.device)
        rb.paged_plan(cached, ints(fresh), self.free, self.table, self.pages, self.page_size, starts, slots, positions,
                      self.used)
        P1, Y = torch.empty_like(X1), torch.empty_like(X1)
        rb.paged_store(X1, X2, I, theta, PAIRING, ROPE_BASE, positions, slots, P1, self.P2, self.I)
        prob = rb.paged_for(P1, self.P2, len(fresh), self.table.shape[1], TAU_S, LAM, rb.RELATION_LAYOUT_BHTD)
        need = rb.relation_paged_workspace_bytes(prob, most)
        if self.workspace is None or self.workspace.numel() < need:
            self.workspace = torch.empty(need, dtype=torch.uint8, device=self.device)
        rb.paged_fwd(P1, self.P2, self.I, self.table, starts, cached, most, TAU_S, LAM, Y=Y, workspace=self.workspace)
        # What the plan took from the front of the free list, from the lengths alone.
        pages = lambda n: -(-n // self.page_size)  # noqa: E731
        taken = sum(pages(c + f) - pages(c) for c, f in zip(self.lengths, fresh))
        self.free = self.free[taken:].contiguous()
        self.lengths = [c + f for c, f in zip(self.lengths, fresh)]
        return Y


def main(prompts=(700, 33, 1, 256, 90), decode=6, chunk=256, heads=8, d_h=64, page_size=64):
    """Serves the prompts; returns the largest difference to the dense path, relative to max |I|."""
    gen = torch.Generator().manual_seed(5)
    total = [p + decode for p in prompts]
    states = [[torch.randn(t, heads, d_h, generator=gen).bfloat16().cuda() for _ in range(3)] for t in total]
    theta = (torch.randn(heads // 2, generator=gen) * 0.3).cuda()
    pages = sum(-(-t // page_size) for t in total) + 3
    cache = PagedCache(len(prompts), heads, d_h, pages, page_size, -(-max(total) // page_size))
    outputs = [[] for _ in prompts]
    steps = 0
    while any(n < t for n, t in zip(cache.lengths, total)):
        # A prompt's next chunk, or one token; requests arrive one step after another.
        fresh = [0 if steps < r else min(chunk, p - n) if n < p else min(1, t - n)
                 for r, (n, p, t) in enumerate(zip(cache.lengths, prompts, total))]
        rows = [[s[n: n + f] for s in st] for st, n, f in zip(states, cache.lengths, fresh)]
        Y = cache.step(*(torch.cat([r[k] for r in rows]) for k in range(3)), theta, fresh)
        for out, part in zip(outputs, Y.split(fresh)):
            out.append(part)
        steps += 1
    torch.cuda.synchronize()
    if rb.relation_check_device_status() != 0:
        raise RuntimeError("a device-side wait expired or an index was out of range")
    worst = 0.0
    for st, out in zip(states, outputs):
        X1, X2, I = (s.transpose(0, 1).unsqueeze(0).contiguous() for s in st)  # [1, heads, T, d_h]
        P1, P2, mixed = (torch.empty_like(X1) for _ in range(3))
        rb.relation_prologue_fwd(rb.problem_for(X1, TAU_S, LAM, True), X1, X2, I, theta, PAIRING, ROPE_BASE, None, P1,
                                 P2, mixed)
        dense, _ = rb.fwd(P1, P2, mixed, TAU_S, LAM, True)
        diff = (torch.cat(out).transpose(0, 1).float() - dense[0].float()).abs().max()
        worst = max(worst, float(diff / mixed.float().abs().max()))
    print(f"{len(prompts)} requests, {sum(total)} tokens in {steps} steps: largest difference to the dense path "
          f"{worst:.1e} of max |I|")
    return worst


if __name__ == "__main__":
    if main() > 2e-2:  # both sides are within 1e-2 of the formula
        sys.exit(1)
