"""The paged forward's cases over 8-bit pages: rows quantised here, in 64 bits, from the bf16 case's pools."""
import numpy as np
import torch

from relation_token_mixing_gb300 import binding as rb
from test_gpu_paged import SENTINEL, Case


def quantised(pool, d, gen):
    """(q, scale, what they stand for) of a pool's rows; rows that are NaN (no token's) get whole numbers of any
    kind and a NaN scale."""
    x = pool[..., :d].double().numpy()
    top = np.abs(x).max(-1)
    dead = ~np.isfinite(top)
    top = np.where(dead, 1.0, top)
    with np.errstate(divide="ignore"):
        s = 2.0 ** np.maximum(np.ceil(np.log2(top / 127)), -126)
    q = np.rint(np.where(dead[..., None], 0, x) / s[..., None])
    q[dead] = torch.randint(-128, 128, q[dead].shape, generator=gen).numpy()
    s = np.where(dead, np.nan, s)
    row = rb.paged_row_q8(d)
    out = torch.randint(-128, 128, (*q.shape[:3], row), generator=gen, dtype=torch.int8)
    out[..., :d] = torch.from_numpy(q).to(torch.int8)
    return out, torch.from_numpy(s).bfloat16(), torch.from_numpy(q * s[..., None])


class Q8Case(Case):
    """A bf16 case whose pages are 8-bit; spread: rows of each token times a power of two of up to 2^+-spread."""

    def __init__(self, *a, spread=0, **kw):
        super().__init__(*a, **kw)
        gen = torch.Generator().manual_seed(77)
        if spread:
            pool = self.pools[1]
            shift = torch.randint(-spread, spread + 1, pool.shape[:3], generator=gen)
            self.pools = (self.pools[0], (pool.double() * 2.0 ** shift.double()[..., None]).bfloat16())
            live = self.pools[1].float()
            self.vmax = float(live[torch.isfinite(live)].abs().max())
        d = self.P1.shape[-1]
        (k, ks, kd), (v, vs, vd) = (quantised(p, d, gen) for p in self.pools)
        self.q8 = k, v, torch.stack([ks, vs], -1)
        self.pools = kd, vd

    def run(self, max_fresh=None, stream=None):
        dev = [x.cuda() for x in (self.P1, *self.q8, self.table, self.starts, self.cached)]
        Y = torch.full_like(dev[0], SENTINEL)
        L = torch.full(self.P1.shape[:2], SENTINEL, device="cuda")
        m = max(f for _, f in self.rows) if max_fresh is None else max_fresh
        prob = rb.paged_q8_for(*self.P1.shape, *dev[1:4], len(self.rows), self.table.shape[1], self.tau, self.lam,
                               self.layout)
        ws = torch.full((rb.relation_paged_q8_workspace_bytes(prob, m) // 4 + 4,), float("nan"), device="cuda")
        torch.cuda.synchronize()
        rb.paged_fwd_q8(*dev, m, self.tau, self.lam, Y, L, ws, self.layout, stream)
        torch.cuda.synchronize()
        return Y.cpu(), L.cpu()
