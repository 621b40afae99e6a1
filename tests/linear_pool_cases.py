"""Inputs, the call and the comparison that the tests of Linear Relation over a pool of states share."""
import numpy as np
import torch

from oracle import linear_pool as lo
from relation_token_mixing_gb300 import binding as rb

TAU = 2.0


def retention(N, H, d, gen, gate, scale=1.0):
    """(G, A_log, dt_bias): log-retentions as the layers have them at the start of training."""
    rate = scale * (1 + 15 * torch.rand(H, d, generator=gen))
    step = torch.exp(torch.empty(H, d).uniform_(-6.9, -2.3, generator=gen))
    bias = torch.log(torch.expm1(step))
    z = 0.5 * torch.randn(N, H, d, generator=gen)
    if gate:
        return z, torch.log(rate), bias
    return -rate * torch.nn.functional.softplus(z + bias), None, None


def inputs(lengths, H, d, gate=False, slots=None, scale=1.0, spare=0, seed=0):
    """Packed tensors of requests of these lengths, `spare` rows behind them; slots: (in, out) lists."""
    gen = torch.Generator().manual_seed(seed)
    R, N = len(lengths), sum(lengths) + spare
    G, A, b = retention(N, H, d, gen, gate, scale)
    P1, P2, I = (torch.randn(N, H, d, generator=gen).bfloat16() for _ in range(3))
    si, so = slots or ([r if r % 3 else -1 for r in range(R)], [R + r for r in range(R)])
    pool = torch.randn(max([R] + [x + 1 for x in si + so]), H, d, d, generator=gen) * 0.5
    starts = [0]
    for n in lengths:
        starts.append(starts[-1] + n)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32)  # noqa: E731
    return dict(P1=P1, P2=P2, I=I, G=G, A_log=A, dt_bias=b, starts=i32(starts), states=pool, slots_in=i32(si),
                slots_out=i32(so))


def on_gpu(x):
    return {k: None if t is None else t.cuda() for k, t in x.items()}


def packed(x, max_fresh=0, **kw):
    return rb.linear_packed_fwd(x["P1"], x["P2"], x["I"], x["G"], x["starts"], x["states"], x["slots_in"],
                                x["slots_out"], max_fresh, TAU, x["A_log"], x["dt_bias"], **kw)


def reference(x):
    a = {k: None if t is None else t.double().numpy() if t.is_floating_point() else t.numpy() for k, t in x.items()}
    args = (a["P1"], a["P2"], a["I"], a["G"], a["starts"], a["states"], a["slots_in"], a["slots_out"], TAU, a["A_log"],
            a["dt_bias"])
    return lo.fwd(*args), lo.fwd(*args, magnitudes=True)


def check(x, Y, states, chunked=True):
    """Y and the pool against the recurrence in 64 bits.

    Y is rounded once to bf16, 2^-8 of itself.  In chunks a weight's two factors and the weight are rounded to bf16, or
    the query's factor and the state, so the sum of magnitudes gives 3 2^-8 of itself; the recurrence rounds in float32:
    with some 8 roundings a token, 2^-18 for the 16 tokens that run in it.
    The state: the key's factor is kept to 2^-24, to 2^-16 in a strongly fading chunk; the sums of log2-retentions, up to 100 in a half chunk, have up to
    16 roundings of 2^-18 each, ln 2 of which is the relative error; together below 2^-14 of the sum of magnitudes.
    A sum's own rounding, and that of small exponentials, stays below 2^-20 of the largest."""
    (Yr, Sr), (Ya, Sa) = reference(x)
    rows = ~np.isnan(Yr)
    got = Y.double().cpu().numpy()
    tol = 2.0 ** -8 * np.abs(Yr) + (3 * 2.0 ** -8 if chunked else 2.0 ** -18) * 1.01 * Ya + 2.0 ** -20
    bad = ~(np.abs(got - Yr)[rows] <= tol[rows])  # (a NaN is no smaller than anything)
    assert not bad.any(), (int(bad.sum()), float((np.abs(got - Yr)[rows] / tol[rows]).max()))
    tol = 2.0 ** -14 * Sa + 2.0 ** -20 * max(1.0, float(Sa.max()))
    off = np.abs(states.double().cpu().numpy() - Sr)
    assert (off <= tol).all(), float((off / tol).max())
