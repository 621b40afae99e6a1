"""Float64 oracle of the paged Relation Cache (TEST INFRASTRUCTURE ONLY).

"Ask Self, Ask Others: Relation Is All You Need", Sec. 5.3 eq.(18) and Appendix A.5
(the cache holds P2 and the information states of the tokens already processed;
a new row forms only its own Relation row), with the cache held in pages that a
block table names.  The plan is written request by request and token by token, the
store row by row, the forward row by row; nothing is shared with the library.
"""
from __future__ import annotations

import math

import numpy as np

BHTD, BTHD = 0, 1


def plan(cached, fresh, free_pages, table, pages: int, page: int, N: int):
    """(table, starts, slots, positions, used) as Python / numpy integers; table is copied."""
    table = np.array(table, dtype=np.int64)
    R, width = table.shape
    starts, used = [0], 0
    slots, positions = [-1] * N, [0] * N
    for r in range(R):
        c, f = int(cached[r]), int(fresh[r])
        for k in range(min(-(-c // page), width), min(-(-(c + f) // page), width)):
            table[r, k] = free_pages[used] if used < len(free_pages) else -1
            used += 1
        for t in range(f):
            n, pos = starts[-1] + t, c + t
            positions[n] = pos
            if pos < width * page and 0 <= table[r, pos // page] < pages:
                slots[n] = int(table[r, pos // page]) * page + pos % page
        starts.append(starts[-1] + f)
    return table, np.array(starts), np.array(slots, dtype=np.int64), np.array(positions), used


def row_of(pages_array, slot: int, g: int, page: int, layout: int):
    """View of the cached row of cache head g at a slot."""
    if layout == BHTD:
        return pages_array[slot // page, g, slot % page]
    return pages_array[slot // page, slot % page, g]


def _turn(x, pos: int, base: float):
    if base <= 0:
        return x.copy()
    half = x.shape[-1] // 2
    a = pos * base ** (-2.0 * np.arange(half) / x.shape[-1])
    lo, hi = x[..., :half], x[..., half:]
    return np.concatenate([np.cos(a) * lo - np.sin(a) * hi, np.sin(a) * lo + np.cos(a) * hi], -1)


def store(X1, X2, I, theta, pairing: int, base: float, positions, slots, P2_pages, I_pages, page: int, layout: int):
    """(P1, P2_pages, I_pages); the pools are copied."""
    X1, X2, I = (np.asarray(x, dtype=np.float64) for x in (X1, X2, I))
    P2_pages, I_pages = (np.array(x, dtype=np.float64) for x in (P2_pages, I_pages))
    N, G, d = X2.shape
    P1 = np.stack([_turn(X1[n], int(positions[n]), base) for n in range(N)]) if N else X1
    for n in range(N):
        if slots[n] < 0:
            continue
        mixed = I[n].copy()
        if theta is not None:
            for k, th in enumerate(theta):
                a, b = 2 * k + pairing, (2 * k + pairing + 1) % G
                mixed[a] = math.cos(th) * I[n, a] - math.sin(th) * I[n, b]
                mixed[b] = math.sin(th) * I[n, a] + math.cos(th) * I[n, b]
        turned = _turn(X2[n], int(positions[n]), base)
        for g in range(G):
            row_of(P2_pages, int(slots[n]), g, page, layout)[:d] = turned[g]
            row_of(I_pages, int(slots[n]), g, page, layout)[:d] = mixed[g]
    return P1, P2_pages, I_pages


def fwd(P1, P2_pages, I_pages, table, starts, cached, tau_S: float, lam: float, page: int, layout: int, only=None):
    """(Y [N, H, d], L [N, H]) of the packed rows that belong to a request (others NaN).
    only: the packed rows wanted (all when None)."""
    P1 = np.asarray(P1, dtype=np.float64)
    N, H, d = P1.shape
    G = P2_pages.shape[1 if layout == BHTD else 2]
    Y, L = np.full((N, H, d), np.nan), np.full((N, H), np.nan)
    wanted = None if only is None else set(int(n) for n in only)
    for r in range(len(cached)):
        rows = [n for n in range(int(starts[r]), int(starts[r + 1])) if wanted is None or n in wanted]
        if not rows:
            continue
        total = int(cached[r]) + int(starts[r + 1]) - int(starts[r])
        ids = np.asarray(table[r][: -(-total // page)], dtype=np.int64)
        for g in range(G):
            if layout == BHTD:
                K, V = (np.asarray(x[ids, g], dtype=np.float64).reshape(-1, x.shape[-1])[:total, :d]
                        for x in (P2_pages, I_pages))
            else:
                K, V = (np.asarray(x[ids, :, g], dtype=np.float64).reshape(-1, x.shape[-1])[:total, :d]
                        for x in (P2_pages, I_pages))
            for n in rows:
                i = int(cached[r]) + n - int(starts[r])
                for h in range(g * (H // G), (g + 1) * (H // G)):
                    U = K[: i + 1] @ P1[n, h] / math.sqrt(d)
                    with np.errstate(over="ignore"):
                        R = U / (1.0 + np.exp(-U)) - lam * math.log(i + 1)
                        R[i] = 1.0 / (1.0 + np.exp(-U[i] / tau_S))
                    m = R.max()
                    w = np.exp(R - m)
                    Y[n, h] = w @ V[: i + 1] / w.sum()
                    L[n, h] = m + math.log(w.sum())
    return Y, L
