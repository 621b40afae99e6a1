"""Float64 oracle of Linear Relation over a pool of states (TEST INFRASTRUCTURE ONLY).

"Ask Self, Ask Others: Relation Is All You Need", Sec. 5.2 eq.(15)-(17) and Appendix A.4: the recurrence token by
token, from the state in one slot of a pool to another.  Written on its own; nothing is shared with the library.
"""
from __future__ import annotations

import math

import numpy as np


def _terms(P1, P2, G, A_log, dt_bias, tau_S):
    """q = S p1^, k = S p2^ and the retention, [N, H, d]."""
    P1, P2, G = (np.asarray(x, dtype=np.float64) for x in (P1, P2, G))
    S = 1.0 / (1.0 + np.exp(-(P1 * P2).sum(-1, keepdims=True) / (tau_S * math.sqrt(P1.shape[-1]))))

    def unit(x):
        n = np.sqrt((x * x).sum(-1, keepdims=True))
        return np.divide(x, n, out=np.zeros_like(x), where=n > 0)

    if A_log is not None:
        G = -np.exp(np.asarray(A_log, dtype=np.float64)) * np.logaddexp(0.0, G + np.asarray(dt_bias, dtype=np.float64))
    with np.errstate(over="ignore", under="ignore"):
        return S * unit(P1), S * unit(P2), np.exp(G)


def fwd(P1, P2, I, G, starts, states, slots_in, slots_out, tau_S, A_log=None, dt_bias=None, magnitudes=False):
    """(Y [N, H, d], states): rows outside the requests' are NaN; the pool is copied.  magnitudes: the same sums of
    absolute values, without the tokens' own states in Y, which the bounds of rounding errors are multiples of."""
    q, k, keep = _terms(P1, P2, G, A_log, dt_bias, tau_S)
    v, old = np.asarray(I, dtype=np.float64), np.asarray(states, dtype=np.float64)
    if magnitudes:
        q, k, v, old = np.abs(q), np.abs(k), np.abs(v), np.abs(old)
    new, Y = old.copy(), np.full(v.shape, np.nan)
    for r in range(len(slots_in)):
        C = old[slots_in[r]].copy() if slots_in[r] >= 0 else np.zeros(old.shape[1:])
        for n in range(int(starts[r]), int(starts[r + 1])):
            C *= keep[n][:, :, None]
            e = np.einsum("hc,hcv->hv", q[n], C)
            Y[n] = e if magnitudes else v[n] + e
            C += k[n][:, :, None] * v[n][:, None, :]
        if slots_out[r] >= 0:
            new[slots_out[r]] = C
    return Y, new
