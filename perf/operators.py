"""Cases of the paged Relation Cache operators: the plan (block tables and slot maps from request lengths), the
store (RoPE, Givens mixing and the scatter of new tokens into pages) and the forward (Relation of a chunk of new
tokens, one or many, over the pages).  Head counts, widths and lengths are those of the repository's own workloads
(8 to 32 heads of 48 to 128, contexts of 1024 to 32768 tokens)."""
import math
import random

import torch

own = False

ROPE_BASE = 1e4
LAYOUTS = {"bhtd": 0, "bthd": 1}
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # the plan of one decoding step of a small serving batch: latency is all of it
        _plan("plan_decode_r64", requests=64, cached=(1, 4096), fresh=(1, 1), page=64, ragged=1),
        # a step of a busy server: decoding requests, idle ones and prompts of all lengths, small pages
        _plan("plan_mixed_r1024", requests=1024, cached=(0, 8192), fresh=(0, 64), page=16, ragged=2),
        # the new token of every request of a decoding batch enters the cache
        _store("store_decode_n64_h16", tokens=64, H=16, G=16, d=64, page=64, ragged=3),
        # a prompt chunk of the widest heads, four relation heads to a cache head, token-major pages
        _store("store_chunk_n16384_h32_g8_d128", tokens=16384, H=32, G=8, d=128, page=64, ragged=4, layout="bthd"),
        # the hybrid model's 60-wide heads, whose rows are no multiple of 16 bytes; an odd number of tokens
        _store("store_odd_n4999_h8_d60", tokens=4999, H=8, G=8, d=60, page=16, ragged=5),
        # decoding with a short history: a few requests, every head with a cache head of its own
        _fwd("decode_r8_h16_d64", requests=8, cached=(500, 4095), fresh=(1, 1), H=16, G=16, d=64, page=64, ragged=6),
        # decoding with long histories of very different lengths, grouped heads
        _fwd("decode_r32_h32_g8_d128", requests=32, cached=(1000, 32767), fresh=(1, 1), H=32, G=8, d=128, page=64,
             ragged=7),
        # drafted tokens to verify: nought to five new tokens a request, large evidence as in late training
        _fwd("few_r48_h10_g5_d64", requests=48, cached=(0, 8192), fresh=(0, 5), H=10, G=5, d=64, page=32, ragged=8,
             spread=True, layout="bthd"),
        # whole prompts packed one after another, of one token to 4096
        _fwd("prompts_r9_h16_d64", requests=9, cached=(0, 0), fresh=(1, 4096), H=16, G=16, d=64, page=128, ragged=9),
        # two prompt chunks over long histories
        _fwd("chunk_r2_h32_g8_d128", requests=2, cached=(15360, 31744), fresh=(1024, 1024), H=32, G=8, d=128, page=64,
             ragged=10),
        # one step of mixed work: mostly decoding, some chunks of a few hundred tokens, 80-wide heads
        _fwd("mixed_r24_h8_g4_d80", requests=24, cached=(100, 8000), fresh=(1, 1), H=8, G=4, d=80, page=16, ragged=11,
             chunks=4, chunk=500),
        # the float32 path: small chunks over small histories
        _fwd("chunk_f32_r4_h16_g8_d64", requests=4, cached=(0, 2048), fresh=(100, 500), H=16, G=8, d=64, page=16,
             ragged=12, dtype="f32"),
    ]


def _plan(name, requests, cached, fresh, page, ragged):
    return {"name": name, "op": "plan", "requests": requests, "cached_lo": cached[0], "cached_hi": cached[1],
            "fresh_lo": fresh[0], "fresh_hi": fresh[1], "chunks": 0, "chunk": 0, "page": page, "ragged": ragged}


def _store(name, tokens, H, G, d, page, ragged, layout="bhtd", dtype="bf16"):
    return {"name": name, "op": "store", "tokens": tokens, "H": H, "G": G, "d": d, "page": page, "ragged": ragged,
            "layout": layout, "dtype": dtype}


def _fwd(name, requests, cached, fresh, H, G, d, page, ragged, layout="bhtd", dtype="bf16", spread=False, chunks=0,
         chunk=0):
    return {"name": name, "op": "fwd", "requests": requests, "cached_lo": cached[0], "cached_hi": cached[1],
            "fresh_lo": fresh[0], "fresh_hi": fresh[1], "chunks": chunks, "chunk": chunk, "H": H, "G": G, "d": d,
            "page": page, "ragged": ragged, "layout": layout, "dtype": dtype, "spread": spread}


def _log_uniform(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    page = rng.choice((16, 32, 64, 128, 256))
    ragged = rng.randrange(1, 1 << 30)
    layout = rng.choice(("bhtd", "bthd"))
    H, G = rng.choice(((8, 8), (8, 4), (10, 10), (10, 5), (12, 12), (12, 4), (16, 16), (16, 2), (32, 8)))
    d = rng.choice((48, 60, 64, 80, 128))
    op = rng.choice(("plan", "store", "fwd", "fwd", "fwd"))
    if op == "plan":
        c = _plan("", _log_uniform(rng, 1, 1024), (0, _log_uniform(rng, 1, 8192)), (rng.randrange(2),
                  _log_uniform(rng, 1, 64)), page, ragged)
    elif op == "store":
        G += G % 2  # mixing pairs the cache heads
        c = _store("", _log_uniform(rng, 1, 16384), H if H % G == 0 else G, G, d, page, ragged, layout,
                   rng.choice(("bf16", "bf16", "f32")))
    else:
        kind = rng.choice(("decode", "few", "chunk", "prompts", "mixed", "f32"))
        if kind == "decode":
            c = _fwd("", _log_uniform(rng, 1, 32), (0, _log_uniform(rng, 16, 32767)), (1, 1), H, G, d, page, ragged,
                     layout, spread=rng.random() < 0.3)
        elif kind == "few":
            c = _fwd("", _log_uniform(rng, 1, 32), (0, _log_uniform(rng, 16, 16384)), (0, rng.randrange(2, 9)), H, G, d,
                     page, ragged, layout, spread=rng.random() < 0.3)
        elif kind == "chunk":
            top = _log_uniform(rng, 16, 16384)
            c = _fwd("", _log_uniform(rng, 1, 4), (top // 2, top), (1, _log_uniform(rng, 16, 1024)), H, G, d, page,
                     ragged, layout, spread=rng.random() < 0.3)
        elif kind == "prompts":
            c = _fwd("", _log_uniform(rng, 1, 8), (0, 0), (1, _log_uniform(rng, 16, 4096)), H, G, d, page, ragged, layout)
        elif kind == "mixed":
            c = _fwd("", _log_uniform(rng, 4, 24), (0, _log_uniform(rng, 256, 8000)), (1, 1), H, G, d, page, ragged,
                     layout, chunks=rng.randrange(1, 4), chunk=_log_uniform(rng, 16, 400))
        else:
            c = _fwd("", _log_uniform(rng, 1, 3), (0, _log_uniform(rng, 16, 1024)), (1, _log_uniform(rng, 1, 300)), H, G,
                     d, page, ragged, layout, dtype="f32")
    del c["name"]
    return c


def _requests(case):
    """(tokens in the cache, new tokens) of each request: the case's own, in an order that the seed shuffles."""
    r = random.Random(case["ragged"])
    rows = [(r.randint(case["cached_lo"], case["cached_hi"]), r.randint(case["fresh_lo"], case["fresh_hi"]))
            for _ in range(case["requests"])]
    rows = [(c, r.randint(max(1, case["chunk"] // 2), case["chunk"]) if k < case["chunks"] else f)
            for k, (c, f) in enumerate(rows)]
    if sum(f for _, f in rows) == 0:
        rows[0] = (rows[0][0], 1)
    if case["cached_lo"] == 0 and case["cached_hi"] == 0 and case["fresh_hi"] > 1:
        rows[0] = (0, case["fresh_hi"])  # whole prompts: the longest one is there, and one of one token
        rows[-1] = rows[-1] if len(rows) == 1 else (0, 1)
    return rows


def _row(case):
    """Elements from one cached row to the next: rows start on 16 bytes."""
    return -(-case["d"] // 8) * 8 if case["dtype"] == "bf16" else case["d"]


def _pages_shape(case, pages):
    if case["layout"] == "bhtd":
        return (pages, case["G"], case["page"], _row(case))
    return (pages, case["page"], case["G"], _row(case))


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = random.Random(seed)

    def normal(*shape, dtype=torch.float32, scale=1.0):
        return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)

    def ints(x, dtype=torch.int32):
        return torch.tensor(x, dtype=dtype, device="cuda")

    s = {"case": case}
    ps = case["page"]
    if case["op"] == "store":
        n, dt, lay = case["tokens"], DTYPES[case["dtype"]], case["layout"]
        lens = random.Random(case["ragged"])
        firsts = [lens.randint(0, 32767 - 64) for _ in range(-(-n // 64))]  # runs of tokens of one request
        r.shuffle(firsts)
        s["positions"] = ints([firsts[i // 64] + i % 64 for i in range(n)])
        pages = -(-n // ps) + 3
        order = torch.randperm(pages, generator=g, device="cuda")
        i = torch.arange(n, device="cuda")
        s["slots"] = order[i // ps] * ps + i % ps
        s |= {"X1": normal(n, case["H"], case["d"], dtype=dt), "X2": normal(n, case["G"], case["d"], dtype=dt),
              "I": normal(n, case["G"], case["d"], dtype=dt), "theta": normal(case["G"] // 2, scale=0.5),
              "P1": torch.empty(n, case["H"], case["d"], dtype=dt, device="cuda"),
              "P2_pages": torch.zeros(_pages_shape(case, pages), dtype=dt, device="cuda"),
              "I_pages": torch.zeros(_pages_shape(case, pages), dtype=dt, device="cuda"), "layout": LAYOUTS[lay]}
        return s
    rows = _requests(case)
    r.shuffle(rows)
    cached, fresh = [c for c, _ in rows], [f for _, f in rows]
    R, N = len(rows), sum(fresh)
    held = [-(-c // ps) for c in cached]
    width = max(-(-(c + f) // ps) for c, f in rows)
    pages = sum(-(-(c + f) // ps) for c, f in rows) + 5
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    s |= {"cached": ints(cached), "fresh": ints(fresh), "tokens": N, "pages": pages, "page": ps, "longest": max(fresh)}
    if case["op"] == "plan":
        # the pages of the cached tokens are there, the free list holds the rest in the order of their release
        k = torch.arange(width, device="cuda")
        h = ints(held, torch.int64)
        at = (torch.cumsum(h, 0) - h)[:, None] + k
        s["block_table"] = torch.where(k < h[:, None], order[at.clamp(max=pages - 1)], torch.full_like(at, -1).int())
        s["free_pages"] = order[sum(held):].contiguous()
        s |= {"starts": torch.empty(R + 1, dtype=torch.int32, device="cuda"),
              "slots": torch.empty(N, dtype=torch.int64, device="cuda"),
              "positions": torch.empty(N, dtype=torch.int32, device="cuda"),
              "used": torch.empty(1, dtype=torch.int32, device="cuda")}
        return s
    dt, H, G, d = DTYPES[case["dtype"]], case["H"], case["G"], case["d"]
    need = ints([-(-(c + f) // ps) for c, f in rows], torch.int64)
    k = torch.arange(width, device="cuda")
    at = (torch.cumsum(need, 0) - need)[:, None] + k
    s["block_table"] = torch.where(k < need[:, None], order[at.clamp(max=pages - 1)], torch.full_like(at, -1).int())
    s["starts"] = ints([0] + [sum(fresh[:i + 1]) for i in range(R)])
    scale = 3.0 / d ** 0.25 if case["spread"] else 1.0
    s |= {"P1": normal(N, H, d, dtype=dt, scale=scale), "P2_pages": normal(*_pages_shape(case, pages), dtype=dt, scale=scale),
          "I_pages": normal(*_pages_shape(case, pages), dtype=dt), "Y": torch.empty(N, H, d, dtype=dt, device="cuda"),
          "layout": LAYOUTS[case["layout"]], "tau_S": 0.5 if case["spread"] else 2.0, "lam": 0.5,
          "workspace": torch.empty(64 << 20, dtype=torch.uint8, device="cuda")}
    return s


def run(s):
    return {"plan": _run_plan, "store": _run_store, "fwd": _run_fwd}[s["case"]["op"]](s)


def _run_plan(s):
    if own:
        from relation_token_mixing_gb300 import binding as rb

        rb.paged_plan(s["cached"], s["fresh"], s["free_pages"], s["block_table"], s["pages"], s["page"], s["starts"],
                      s["slots"], s["positions"], s["used"])
        return [s["block_table"], s["starts"], s["slots"], s["positions"], s["used"]]
    ps, table, free = s["page"], s["block_table"], s["free_pages"]
    R, W = table.shape
    held = torch.clamp((s["cached"] + ps - 1) // ps, max=W)
    need = torch.clamp((s["cached"] + s["fresh"] + ps - 1) // ps, max=W)
    new = need - held
    ends = torch.cumsum(s["fresh"], 0).int()
    starts = torch.cat([ends.new_zeros(1), ends])
    k = torch.arange(W, device=table.device)
    nth = (torch.cumsum(new, 0) - new)[:, None] + k - held[:, None]
    ids = torch.where(nth < free.numel(), free[nth.clamp(0, max(free.numel() - 1, 0))] if free.numel() else table, -1)
    table.copy_(torch.where((k >= held[:, None]) & (k < need[:, None]), ids, table))
    token = torch.arange(s["tokens"], dtype=torch.int32, device=table.device)
    r = torch.searchsorted(ends, token, right=True).clamp(max=R - 1)
    known = token < ends[-1]
    pos = torch.where(known, s["cached"][r] + token - starts[r], 0)
    page = table[r, (pos // ps).clamp(max=W - 1)].long()
    slots = torch.where(known & (pos < W * ps) & (page >= 0) & (page < s["pages"]), page * ps + pos % ps, -1)
    return [table, starts, slots, pos.int(), new.sum().int().reshape(1)]


def _turned(x, positions):
    """RoPE in its half-split form: columns c and c + d/2 turn by positions * base^(-2c/d)."""
    half = x.shape[-1] // 2
    # the angle in turns, as a fraction with 44 bits, so that large positions keep it
    f = torch.tensor([round(ROPE_BASE ** (-c / half) / (2 * math.pi) * 2 ** 44) for c in range(half)], device=x.device)
    part = (positions.long()[:, None] * f) & ((1 << 44) - 1)
    angle = part.float() * (2 * math.pi / 2 ** 44)
    cs, sn = torch.cos(angle)[:, None], torch.sin(angle)[:, None]
    a, b = x[..., :half], x[..., half:]
    return torch.cat([cs * a - sn * b, sn * a + cs * b], -1)


def _rows_of(pages, slots, page, layout):
    """The cached rows [tokens, G, row] of some slots, as (index, view) for reading and writing."""
    return (slots // page, slice(None), slots % page) if layout == 0 else (slots // page, slots % page)


def _run_store(s):
    c = s["case"]
    if own:
        from relation_token_mixing_gb300 import binding as rb

        rb.paged_store(s["X1"], s["X2"], s["I"], s["theta"], 0, ROPE_BASE, s["positions"], s["slots"], s["P1"],
                       s["P2_pages"], s["I_pages"], s["layout"])
        return [s["P1"], s["P2_pages"], s["I_pages"]]
    dt, d = s["X1"].dtype, c["d"]
    i = s["I"].float()
    cs, sn = torch.cos(s["theta"])[:, None], torch.sin(s["theta"])[:, None]
    a, b = i[:, 0::2], i[:, 1::2]
    mixed = torch.stack([cs * a - sn * b, sn * a + cs * b], 2).flatten(1, 2)
    at = _rows_of(s["P2_pages"], s["slots"], c["page"], s["layout"])
    s["P2_pages"][..., :d][at] = _turned(s["X2"].float(), s["positions"]).to(dt)
    s["I_pages"][..., :d][at] = mixed.to(dt)
    return [_turned(s["X1"].float(), s["positions"]).to(dt), s["P2_pages"], s["I_pages"]]


def _run_fwd(s):
    c = s["case"]
    if own:
        from relation_token_mixing_gb300 import binding as rb

        rb.paged_fwd(s["P1"], s["P2_pages"], s["I_pages"], s["block_table"], s["starts"], s["cached"], s["longest"],
                     s["tau_S"], s["lam"], s["Y"], None, s["workspace"], s["layout"])
        return [s["Y"]]
    H, G, d, T = c["H"], c["G"], c["d"], s["longest"]
    starts, cached, table = s["starts"].long(), s["cached"].long(), s["block_table"].long().clamp(min=0)
    R = table.shape[0]

    def history(pages):  # [R, G, tokens, d]
        x = pages[table]
        x = x.permute(0, 2, 1, 3, 4) if s["layout"] == 0 else x.permute(0, 3, 1, 2, 4)
        return x.flatten(2, 3)[..., :d].float()

    fresh = starts[1:] - starts[:-1]
    t = torch.arange(T, device=table.device)
    rows = (starts[:-1, None] + t).clamp(max=s["P1"].shape[0] - 1)
    q = s["P1"].float()[rows].view(R, T, G, H // G, d).permute(0, 2, 3, 1, 4).reshape(R, G, H // G * T, d)
    u = torch.matmul(q, history(s["P2_pages"]).transpose(2, 3)).mul_(1 / math.sqrt(d)).view(R, G, H // G, T, -1)
    pos = (cached[:, None] + t)[:, None, None, :, None]
    j = torch.arange(u.shape[-1], device=table.device)
    e = u * torch.sigmoid(u) - s["lam"] * torch.log((pos + 1).float())
    own_entry = torch.sigmoid(u.div_(s["tau_S"]))
    e = torch.where(j == pos, own_entry, e)
    del u, own_entry
    e.masked_fill_(j > pos, -math.inf)
    e.sub_(e.amax(-1, keepdim=True)).exp_()
    y = torch.matmul(e.view(R, G, H // G * T, -1), history(s["I_pages"])).view(R, G, H // G, T, d)
    y = y / e.sum(-1, keepdim=True)
    y = y.permute(0, 3, 1, 2, 4).reshape(R, T, H, d)
    return [y[t < fresh[:, None]].to(s["P1"].dtype)]


def work(case):
    e = 4 if case.get("dtype") == "f32" else 2
    if case["op"] == "plan":
        rows = _requests(case)
        ps = case["page"]
        new = sum(-(-(c + f) // ps) - -(-c // ps) for c, f in rows)
        # lengths and the taken free pages in; starts, new table entries, slots and positions out
        return {"bytes": 8 * len(rows) + 4 * (len(rows) + 1) + 8 * new + 12 * sum(f for _, f in rows), "flops": 0}
    if case["op"] == "store":
        n, wide = case["tokens"], case["H"] + 2 * case["G"]
        # three products and sums for each element turned or mixed
        return {"bytes": n * (2 * wide * case["d"] * e + 12), "flops": 3 * n * wide * case["d"]}
    rows = _requests(case)
    n = sum(f for _, f in rows)
    visible = sum(f * c + f * (f + 1) // 2 for c, f in rows)
    history = sum(c + f for c, f in rows if f)
    return {"bytes": (2 * n * case["H"] + 2 * history * case["G"]) * case["d"] * e, "flops": 4 * case["d"] * case["H"] * visible}


def exact(case, seed):
    if case["op"] == "plan":
        return None  # whole numbers only
    s = prepare(case, seed)
    if case["op"] == "store":
        half = case["d"] // 2
        freq = torch.tensor([ROPE_BASE ** (-2.0 * c / case["d"]) for c in range(half)], dtype=torch.float64, device="cuda")
        z = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), s["positions"].double()[:, None] * freq)

        def rope(x):
            w = torch.complex(x[..., :half].double(), x[..., half:].double()) * z[:, None]
            return torch.cat([w.real, w.imag], -1)

        out = [rope(s["X1"]), s["P2_pages"].double(), s["I_pages"].double()]
        mixed = s["I"].double()
        pair = torch.complex(mixed[:, 0::2], mixed[:, 1::2]) * torch.polar(torch.ones_like(s["theta"].double()),
                                                                           s["theta"].double())[None, :, None]
        mixed[:, 0::2], mixed[:, 1::2] = pair.real, pair.imag
        for pages, x in ((out[1], rope(s["X2"])), (out[2], mixed)):
            heads = pages if s["layout"] == 1 else pages.transpose(1, 2)
            heads[s["slots"] // case["page"], s["slots"] % case["page"], :, :case["d"]] = x
        return out
    if 4.0 * case["d"] * case["H"] * sum(f * (c + f) for c, f in _requests(case)) > 4e12:
        return None
    d, group = case["d"], case["H"] // case["G"]
    Y = torch.empty(s["P1"].shape, dtype=torch.float64, device="cuda")
    starts, cached = s["starts"].tolist(), s["cached"].tolist()
    for r, c in enumerate(cached):
        f = starts[r + 1] - starts[r]
        if f == 0:
            continue
        ids = s["block_table"][r, :-(-(c + f) // case["page"])].long()
        i = torch.arange(c, c + f, device="cuda")[:, None]
        j = torch.arange(c + f, device="cuda")[None, :]
        for h in range(case["G"]):
            k, v = ((x[ids, h] if s["layout"] == 0 else x[ids, :, h]).reshape(-1, x.shape[-1])[:c + f, :d].double()
                    for x in (s["P2_pages"], s["I_pages"]))
            for m in range(h * group, (h + 1) * group):
                u = s["P1"][starts[r]:starts[r + 1], m].double() @ k.T / math.sqrt(d)
                w = u / (1 + torch.exp(-u)) - s["lam"] * torch.log((i + 1).double())
                w = torch.where(i == j, 1 / (1 + torch.exp(-u / s["tau_S"])), w)
                w = torch.exp(torch.where(j > i, -math.inf, w) - torch.where(j > i, -math.inf, w).max(1, keepdim=True).values)
                Y[starts[r]:starts[r + 1], m] = (w @ v) / w.sum(1, keepdim=True)
    return [Y]
