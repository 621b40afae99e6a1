"""Cases of the operators that serve the hybrid model's layers: the paged Relation Cache in 8 bits (the store that
quantises rows as it writes them and reads them back, the forward of new tokens over such pages) and Linear Relation
over a pool of states (one token per request in the recurrent form, packed requests of any lengths in the chunked form).
Head counts, widths and lengths are those of the repository's own workloads (8 to 32 heads of 48 to 128, Linear
Relation 8 to 16 heads of 48 to 64, contexts of 1024 to 32768 tokens)."""
import math
import random

import torch

own = False

ROPE_BASE = 1e4
TAU = 2.0
LAYOUTS = {"bhtd": 0, "bthd": 1}


def listed():
    return [
        # a prompt chunk of the widest heads enters the cache, token-major pages, and is read back (a prefix to export)
        _store("store_chunk_n16384_h32_g8_d128", tokens=16384, H=32, G=8, d=128, page=64, ragged=1, layout="bthd"),
        # the hybrid model's 60-wide heads, whose rows are padded in the pages; an odd number of tokens
        _store("store_odd_n4999_h8_d60", tokens=4999, H=8, G=8, d=60, page=16, ragged=2),
        # decoding with a short history: a few requests, every head with a cache head of its own
        _fwd("decode_r8_h16_d64", requests=8, cached=(500, 4095), fresh=(1, 1), H=16, G=16, d=64, page=64, ragged=3),
        # decoding with long histories of very different lengths, grouped heads
        _fwd("decode_r32_h32_g8_d128", requests=32, cached=(1000, 32767), fresh=(1, 1), H=32, G=8, d=128, page=64,
             ragged=4),
        # drafted tokens to verify: nought to five new tokens a request, large evidence as in late training
        _fwd("few_r48_h10_g5_d64", requests=48, cached=(0, 8192), fresh=(0, 5), H=10, G=5, d=64, page=32, ragged=5,
             spread=True, layout="bthd"),
        # two prompt chunks over long histories
        _fwd("chunk_r2_h32_g8_d128", requests=2, cached=(15360, 31744), fresh=(1024, 1024), H=32, G=8, d=128, page=64,
             ragged=6),
        # one step of mixed work: mostly decoding, some chunks of a few hundred tokens, the hybrid model's heads
        _fwd("mixed_r24_h8_d60", requests=24, cached=(100, 8000), fresh=(1, 1), H=8, G=8, d=60, page=16, ragged=7,
             chunks=4, chunk=500),
        # a decoding step of a small batch through one Linear layer of the hybrid model: latency is most of it
        _step("step_r16_h8_d60", requests=16, H=8, d=60, gate=True, ragged=8),
        # a decoding step of a busy server
        _step("step_r512_h16_d64", requests=512, H=16, d=64, gate=False, ragged=9),
        # prompts of all lengths, one after another, new requests and ones that go on from a kept state
        _packed("prompts_r24_h8_d60", requests=24, fresh=(1, 2048), H=8, d=60, gate=True, ragged=10),
        # one long context
        _packed("long_r1_h8_d60", requests=1, fresh=(32768, 32768), H=8, d=60, gate=False, ragged=11),
        # one step of mixed work: mostly decoding, some chunks of a few hundred tokens
        _packed("mixed_r64_h16_d64", requests=64, fresh=(1, 1), H=16, d=64, gate=True, ragged=12, chunks=4, chunk=500),
    ]


def _store(name, tokens, H, G, d, page, ragged, layout="bhtd"):
    return {"name": name, "op": "store", "tokens": tokens, "H": H, "G": G, "d": d, "page": page, "ragged": ragged,
            "layout": layout}


def _fwd(name, requests, cached, fresh, H, G, d, page, ragged, layout="bhtd", spread=False, chunks=0, chunk=0):
    return {"name": name, "op": "fwd", "requests": requests, "cached_lo": cached[0], "cached_hi": cached[1],
            "fresh_lo": fresh[0], "fresh_hi": fresh[1], "chunks": chunks, "chunk": chunk, "H": H, "G": G, "d": d,
            "page": page, "ragged": ragged, "layout": layout, "spread": spread}


def _step(name, requests, H, d, gate, ragged):
    return {"name": name, "op": "step", "requests": requests, "H": H, "d": d, "gate": gate, "ragged": ragged}


def _packed(name, requests, fresh, H, d, gate, ragged, chunks=0, chunk=0):
    return {"name": name, "op": "packed", "requests": requests, "cached_lo": 0, "cached_hi": 0, "fresh_lo": fresh[0],
            "fresh_hi": fresh[1], "chunks": chunks, "chunk": chunk, "H": H, "d": d, "gate": gate, "ragged": ragged}


def _log_uniform(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    ragged = rng.randrange(1, 1 << 30)
    op = rng.choice(("store", "fwd", "fwd", "fwd", "step", "packed", "packed"))
    if op in ("store", "fwd"):
        page = rng.choice((16, 32, 64, 128, 256))
        layout = rng.choice(("bhtd", "bthd"))
        H, G = rng.choice(((8, 8), (8, 4), (10, 10), (10, 5), (12, 12), (12, 4), (16, 16), (16, 2), (32, 8)))
        d = rng.choice((48, 60, 64, 80, 128))
        if op == "store":
            G += G % 2  # mixing pairs the cache heads
            c = _store("", _log_uniform(rng, 1, 16384), H if H % G == 0 else G, G, d, page, ragged, layout)
        else:
            kind = rng.choice(("decode", "few", "chunk", "prompts", "mixed"))
            if kind == "decode":
                c = _fwd("", _log_uniform(rng, 1, 32), (0, _log_uniform(rng, 16, 32767)), (1, 1), H, G, d, page, ragged,
                         layout, spread=rng.random() < 0.3)
            elif kind == "few":
                c = _fwd("", _log_uniform(rng, 1, 32), (0, _log_uniform(rng, 16, 16384)), (0, rng.randrange(2, 9)), H, G,
                         d, page, ragged, layout, spread=rng.random() < 0.3)
            elif kind == "chunk":
                top = _log_uniform(rng, 16, 16384)
                c = _fwd("", _log_uniform(rng, 1, 4), (top // 2, top), (1, _log_uniform(rng, 16, 1024)), H, G, d, page,
                         ragged, layout, spread=rng.random() < 0.3)
            elif kind == "prompts":
                c = _fwd("", _log_uniform(rng, 1, 8), (0, 0), (1, _log_uniform(rng, 16, 4096)), H, G, d, page, ragged,
                         layout)
            else:
                c = _fwd("", _log_uniform(rng, 4, 24), (0, _log_uniform(rng, 256, 8000)), (1, 1), H, G, d, page, ragged,
                         layout, chunks=rng.randrange(1, 4), chunk=_log_uniform(rng, 16, 400))
    else:
        H, d, gate = rng.choice((8, 10, 12, 16)), rng.choice((48, 60, 64)), rng.random() < 0.5
        if op == "step":
            c = _step("", _log_uniform(rng, 1, 512), H, d, gate, ragged)
        else:
            kind = rng.choice(("prompts", "long", "mixed"))
            if kind == "prompts":
                c = _packed("", _log_uniform(rng, 1, 24), (0, _log_uniform(rng, 4, 2048)), H, d, gate, ragged)
            elif kind == "long":
                top = _log_uniform(rng, 512, 16384)
                c = _packed("", rng.randrange(1, 3), (top // 2, top), H, d, gate, ragged)
            else:
                c = _packed("", _log_uniform(rng, 4, 64), (1, 1), H, d, gate, ragged, chunks=rng.randrange(1, 4),
                            chunk=_log_uniform(rng, 8, 800))
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
    if case["cached_hi"] == 0 and case["fresh_hi"] > 1:
        rows[0] = (0, case["fresh_hi"])  # whole prompts: the longest one is there, and one of one token
        rows[-1] = rows[-1] if len(rows) == 1 else (0, 1)
    return rows


def _row(d):
    """Bytes from one cached row to the next: rows start on 16 bytes."""
    return -(-d // 16) * 16


def _pages_shape(case, pages, row):
    if case["layout"] == "bhtd":
        return (pages, case["G"], case["page"], row)
    return (pages, case["page"], case["G"], row)


def _quantised(x):
    """Rows of whole numbers up to 127 and the scale of each, the least power of two (2^-126 at least) that holds it."""
    top = x.abs().amax(-1, keepdim=True)
    m, e = torch.frexp(top / 127)
    k = torch.where(m == 0.5, e - 1, e).clamp(-126, 127)  # top / 127 = m 2^e with m in [0.5, 1)
    scale = torch.where(top > 0, torch.ldexp(torch.ones_like(top), k), torch.full_like(top, 2.0 ** -126))
    q = torch.round(x / scale).clamp(-127, 127).to(torch.int8)
    return q, scale.squeeze(-1).to(torch.bfloat16)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = random.Random(seed)

    def normal(*shape, dtype=torch.float32, scale=1.0):
        return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)

    def uniform(*shape):
        return torch.rand(shape, generator=g, device="cuda")

    def ints(x, dtype=torch.int32):
        return torch.tensor(x, dtype=dtype, device="cuda")

    s = {"case": case}
    bf = torch.bfloat16
    if case["op"] == "store":
        n, d, ps = case["tokens"], case["d"], case["page"]
        lens = random.Random(case["ragged"])
        firsts = [lens.randint(0, 32767 - 64) for _ in range(-(-n // 64))]  # runs of tokens of one request
        r.shuffle(firsts)
        s["positions"] = ints([firsts[i // 64] + i % 64 for i in range(n)])
        pages = -(-n // ps) + 3
        order = torch.randperm(pages, generator=g, device="cuda")
        i = torch.arange(n, device="cuda")
        s["slots"] = order[i // ps] * ps + i % ps
        s |= {"X1": normal(n, case["H"], d, dtype=bf), "X2": normal(n, case["G"], d, dtype=bf),
              "I": normal(n, case["G"], d, dtype=bf), "theta": normal(case["G"] // 2, scale=0.5),
              "P1": torch.empty(n, case["H"], d, dtype=bf, device="cuda"),
              "P2_rows": torch.empty(n, case["G"], d, dtype=bf, device="cuda"),
              "I_rows": torch.empty(n, case["G"], d, dtype=bf, device="cuda"), "layout": LAYOUTS[case["layout"]]}
        for name in ("P2_pages", "I_pages"):
            s[name] = torch.zeros(_pages_shape(case, pages, _row(d)), dtype=torch.int8, device="cuda")
        s["scales"] = torch.zeros(_pages_shape(case, pages, 2), dtype=bf, device="cuda")
        return s
    if case["op"] in ("step", "packed"):
        H, d, R = case["H"], case["d"], case["requests"]
        fresh = [1] * R if case["op"] == "step" else [f for _, f in _requests(case)]
        r.shuffle(fresh)
        N = sum(fresh)
        # retention as the layers have it: exp(A_log) over 1 .. 16, step sizes over 0.001 .. 0.1
        rate = 1 + 15 * uniform(H, d)
        bias = torch.log(torch.expm1(torch.exp(math.log(1e-3) + math.log(100.0) * uniform(H, d))))
        z = normal(N, H, d, scale=0.5)
        s |= {"P1": normal(N, H, d, dtype=bf), "P2": normal(N, H, d, dtype=bf), "I": normal(N, H, d, dtype=bf),
              "G": z if case["gate"] else -rate * torch.nn.functional.softplus(z + bias),
              "A_log": torch.log(rate) if case["gate"] else None, "dt_bias": bias if case["gate"] else None,
              "states": normal(2 * R, H, d, d, scale=0.5), "Y": torch.empty(N, H, d, dtype=bf, device="cuda")}
        # each request goes from one slot of the pool to another; where requests come new, some have no state yet
        order = torch.randperm(2 * R, generator=g, device="cuda").int()
        new = torch.tensor([case["op"] == "packed" and k % 3 == 0 for k in range(R)], device="cuda")
        s |= {"slots_in": torch.where(new, -1, order[:R]).int(), "slots_out": order[R:].contiguous(),
              "fresh": ints(fresh), "starts": ints([0] + [sum(fresh[:k + 1]) for k in range(R)]), "longest": max(fresh),
              "chunks": sum(-(-f // CHUNK) for f in fresh),
              "workspace": torch.empty(256 << 20, dtype=torch.uint8, device="cuda")}
        return s
    ps = case["page"]
    rows = _requests(case)
    r.shuffle(rows)
    cached, fresh = [c for c, _ in rows], [f for _, f in rows]
    R, N = len(rows), sum(fresh)
    width = max(-(-(c + f) // ps) for c, f in rows)
    pages = sum(-(-(c + f) // ps) for c, f in rows) + 5
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    need = ints([-(-(c + f) // ps) for c, f in rows], torch.int64)
    k = torch.arange(width, device="cuda")
    at = (torch.cumsum(need, 0) - need)[:, None] + k
    s["block_table"] = torch.where(k < need[:, None], order[at.clamp(max=pages - 1)], torch.full_like(at, -1).int())
    s["starts"] = ints([0] + [sum(fresh[:i + 1]) for i in range(R)])
    H, G, d = case["H"], case["G"], case["d"]
    scale = 3.0 / d ** 0.25 if case["spread"] else 1.0
    scales = []
    for name, x in (("P2_pages", scale), ("I_pages", 1.0)):
        s[name] = torch.zeros(_pages_shape(case, pages, _row(d)), dtype=torch.int8, device="cuda")
        for lo in range(0, pages, 1024):  # in parts: the rows before they are quantised are four times as large
            part = s[name][lo:lo + 1024]
            q, sc = _quantised(normal(*part.shape[:3], d, scale=x))
            part[..., :d] = q
            scales.append(sc)
    half = len(scales) // 2
    s["scales"] = torch.stack([torch.cat(scales[:half]), torch.cat(scales[half:])], -1)
    s |= {"cached": ints(cached), "longest": max(fresh), "P1": normal(N, H, d, dtype=bf, scale=scale),
          "Y": torch.empty(N, H, d, dtype=bf, device="cuda"), "layout": LAYOUTS[case["layout"]],
          "tau_S": 0.5 if case["spread"] else TAU, "lam": 0.5,
          "workspace": torch.empty(64 << 20, dtype=torch.uint8, device="cuda")}
    return s


def run(s):
    return {"store": _run_store, "fwd": _run_fwd, "step": _run_step, "packed": _run_packed}[s["case"]["op"]](s)


def _turned(x, positions):
    """RoPE in its half-split form: columns c and c + d/2 turn by positions * base^(-2c/d)."""
    half = x.shape[-1] // 2
    c = torch.arange(half, dtype=torch.float64, device=x.device)
    angle = positions.double()[:, None] * ROPE_BASE ** (-c / half)  # far positions keep their angle in 64 bits
    cs, sn = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    a, b = x[..., :half], x[..., half:]
    return torch.cat([cs * a - sn * b, sn * a + cs * b], -1)


def _rows_of(slots, page, layout):
    """The cached rows [tokens, G, row] of some slots, as an index into the pages."""
    return (slots // page, slice(None), slots % page) if layout == 0 else (slots // page, slots % page)


def _run_store(s):
    c = s["case"]
    if own:
        from relation_token_mixing_gb300 import binding as rb

        rb.paged_store_q8(s["X1"], s["X2"], s["I"], s["theta"], 0, ROPE_BASE, s["positions"], s["slots"], s["P1"],
                          s["P2_pages"], s["I_pages"], s["scales"], s["layout"])
        rb.paged_read_q8(s["slots"], s["P2_pages"], s["I_pages"], s["scales"], c["d"], s["P2_rows"], s["I_rows"],
                         s["layout"])
        return [s["P1"], s["P2_rows"], s["I_rows"]]
    d = c["d"]
    i = s["I"].float()
    cs, sn = torch.cos(s["theta"])[:, None], torch.sin(s["theta"])[:, None]
    a, b = i[:, 0::2], i[:, 1::2]
    mixed = torch.stack([cs * a - sn * b, sn * a + cs * b], 2).flatten(1, 2)
    at = _rows_of(s["slots"], c["page"], s["layout"])
    (q2, s2), (qi, si) = _quantised(_turned(s["X2"].float(), s["positions"])), _quantised(mixed)
    s["P2_pages"][..., :d][at] = q2
    s["I_pages"][..., :d][at] = qi
    s["scales"][at] = torch.stack([s2, si], -1)
    held = s["scales"][at].float()
    return [_turned(s["X1"].float(), s["positions"]).bfloat16(),
            (s["P2_pages"][..., :d][at].float() * held[..., :1]).bfloat16(),
            (s["I_pages"][..., :d][at].float() * held[..., 1:]).bfloat16()]


def _run_fwd(s):
    c = s["case"]
    if own:
        from relation_token_mixing_gb300 import binding as rb

        rb.paged_fwd_q8(s["P1"], s["P2_pages"], s["I_pages"], s["scales"], s["block_table"], s["starts"], s["cached"],
                        s["longest"], s["tau_S"], s["lam"], s["Y"], None, s["workspace"], s["layout"])
        return [s["Y"]]
    H, G, d, T = c["H"], c["G"], c["d"], s["longest"]
    starts, cached, table = s["starts"].long(), s["cached"].long(), s["block_table"].long().clamp(min=0)
    R = table.shape[0]

    def history(pages, which):  # [R, G, tokens, d]
        x = pages[table][..., :d].float() * s["scales"][table][..., which, None].float()
        x = x.permute(0, 2, 1, 3, 4) if s["layout"] == 0 else x.permute(0, 3, 1, 2, 4)
        return x.flatten(2, 3)

    fresh = starts[1:] - starts[:-1]
    t = torch.arange(T, device=table.device)
    rows = (starts[:-1, None] + t).clamp(max=s["P1"].shape[0] - 1)
    q = s["P1"].float()[rows].view(R, T, G, H // G, d).permute(0, 2, 3, 1, 4).reshape(R, G, H // G * T, d)
    u = torch.matmul(q, history(s["P2_pages"], 0).transpose(2, 3)).mul_(1 / math.sqrt(d)).view(R, G, H // G, T, -1)
    pos = (cached[:, None] + t)[:, None, None, :, None]
    j = torch.arange(u.shape[-1], device=table.device)
    e = u * torch.sigmoid(u) - s["lam"] * torch.log((pos + 1).float())
    own_entry = torch.sigmoid(u.div_(s["tau_S"]))
    e = torch.where(j == pos, own_entry, e)
    del u, own_entry
    e.masked_fill_(j > pos, -math.inf)
    e.sub_(e.amax(-1, keepdim=True)).exp_()
    y = torch.matmul(e.view(R, G, H // G * T, -1), history(s["I_pages"], 1)).view(R, G, H // G, T, d)
    y = y / e.sum(-1, keepdim=True)
    y = y.permute(0, 3, 1, 2, 4).reshape(R, T, H, d)
    return [y[t < fresh[:, None]].bfloat16()]


def _reads(s):
    """(q, k, v, g) of Linear Relation: S p1^, S p2^, I and the log-retention, [tokens, H, d] in 32 bits."""
    p1, p2 = s["P1"].float(), s["P2"].float()
    n1, n2 = (x.square().sum(-1, keepdim=True).sqrt() for x in (p1, p2))
    S = torch.sigmoid((p1 * p2).sum(-1, keepdim=True) / (TAU * math.sqrt(p1.shape[-1])))
    g = s["G"]
    if s["A_log"] is not None:
        x = g + s["dt_bias"]
        g = -torch.exp(s["A_log"]) * (x.clamp(min=0) + torch.log1p(torch.exp(-x.abs())))
    return S * p1 / n1, S * p2 / n2, s["I"].float(), g


def _entering(s):
    """The state [R, H, d, d] that each request goes on from."""
    return torch.where((s["slots_in"] >= 0)[:, None, None, None], s["states"][s["slots_in"].clamp(min=0).long()], 0.0)


def _run_step(s):
    if own:
        from relation_token_mixing_gb300 import binding as rb

        rb.linear_step(s["P1"], s["P2"], s["I"], s["G"], s["states"], s["slots_in"], s["slots_out"], TAU, s["A_log"],
                       s["dt_bias"], s["Y"])
        return [s["Y"], s["states"]]
    q, k, v, g = _reads(s)
    C = _entering(s) * torch.exp(g)[..., None]
    y = v + torch.matmul(q[..., None, :], C).squeeze(-2)
    s["states"][s["slots_out"].long()] = C + k[..., None] * v[..., None, :]
    return [y.bfloat16(), s["states"]]


CHUNK = 16  # tokens of a chunk of the plain form


def _run_packed(s):
    if own:
        from relation_token_mixing_gb300 import binding as rb

        rb.linear_packed_fwd(s["P1"], s["P2"], s["I"], s["G"], s["starts"], s["states"], s["slots_in"], s["slots_out"],
                             s["longest"], TAU, s["A_log"], s["dt_bias"], s["Y"], s["workspace"])
        return [s["Y"], s["states"]]
    # every request in chunks of its own, all chunks in one list; rows past a request's end do nothing
    fresh, starts, M, dev = s["fresh"].long(), s["starts"].long(), s["chunks"], s["P1"].device
    per = (fresh + CHUNK - 1) // CHUNK
    ends = torch.cumsum(per, 0)
    c = torch.arange(M, device=dev)
    r = torch.searchsorted(ends, c, right=True)
    nth = c - (ends - per)[r]
    t = nth[:, None] * CHUNK + torch.arange(CHUNK, device=dev)
    there = t < fresh[r][:, None]
    rows = (starts[r][:, None] + t).clamp(max=s["P1"].shape[0] - 1)
    q, k, v, g = (torch.where(there[..., None, None], x[rows], 0.0).transpose(1, 2) for x in _reads(s))  # [M, H, 16, d]
    G = torch.cumsum(g, 2)
    i = torch.arange(CHUNK, device=dev)
    D = (G[..., :, None, :] - G[..., None, :, :]).masked_fill_((i[:, None] <= i)[..., None], -math.inf).exp_()
    A = torch.einsum("mhic,mhjc,mhijc->mhij", q, k, D)
    del D
    # the state after each chunk: h <- a h + b, in log2(M) doublings; a chunk that begins a request takes nothing from
    # the one before it
    h = torch.matmul((k * torch.exp(G[:, :, -1:] - G)).transpose(2, 3), v)
    a = torch.exp(G[:, :, -1])[..., None]
    begins = nth == 0
    first = _entering(s)[r[begins]]
    h[begins] += a[begins] * first
    a = torch.where(begins[:, None, None, None], 0.0, a)
    for n in (1 << x for x in range((M - 1).bit_length())):
        h = torch.cat([h[:n], h[n:] + a[n:] * h[:-n]])
        a = torch.cat([a[:n], a[n:] * a[:-n]])
    before = torch.cat([h[:1], h[:-1]])
    before[begins] = first
    y = v + torch.matmul(A, v) + torch.matmul(q * torch.exp(G), before)
    some = fresh > 0
    s["states"][s["slots_out"][some].long()] = h[(ends - 1)[some]]
    s["states"][s["slots_out"][~some].long()] = _entering(s)[~some]  # no new token: the state as it is
    return [y.transpose(1, 2)[there].bfloat16(), s["states"]]


def work(case):
    if case["op"] == "store":
        n, H, G, d = case["tokens"], case["H"], case["G"], case["d"]
        # states in, P1 and the quantised rows with their scales out, and those rows read back; three operations for each
        # element turned or mixed, three to quantise one, one to read it
        return {"bytes": n * ((2 * H + 2 * G) * d * 2 + 4 * G * (d + 2) + 2 * G * d * 2 + 12),
                "flops": n * d * (3 * (H + 2 * G) + 8 * G)}
    H, d = case["H"], case["d"]
    if case["op"] == "step":
        R = case["requests"]
        return {"bytes": R * H * (8 * d * d + 12 * d) + 8 * R, "flops": 5 * d * d * R * H}
    rows = _requests(case)
    n = sum(f for _, f in rows)
    if case["op"] == "packed":
        kept = sum(k % 3 != 0 for k in range(len(rows)))
        return {"bytes": n * H * 12 * d + (kept + len(rows)) * H * d * d * 4, "flops": 5 * d * d * n * H}
    visible = sum(f * c + f * (f + 1) // 2 for c, f in rows)
    history = sum(c + f for c, f in rows if f)
    return {"bytes": 4 * n * H * d + 2 * history * case["G"] * (d + 2), "flops": 4 * d * H * visible}


def exact(case, seed):
    s = prepare(case, seed)
    d = case["d"]
    if case["op"] == "store":
        half = d // 2
        freq = torch.tensor([ROPE_BASE ** (-2.0 * c / d) for c in range(half)], dtype=torch.float64, device="cuda")
        z = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), s["positions"].double()[:, None] * freq)

        def rope(x):
            w = torch.complex(x[..., :half].double(), x[..., half:].double()) * z[:, None]
            return torch.cat([w.real, w.imag], -1)

        def held(x):
            step = torch.exp2(torch.ceil(torch.log2(x.abs().max(-1, keepdim=True).values / 127)))
            return torch.round(x / step) * step

        mixed = s["I"].double()
        pair = torch.complex(mixed[:, 0::2], mixed[:, 1::2]) * torch.polar(torch.ones_like(s["theta"].double()),
                                                                           s["theta"].double())[None, :, None]
        mixed[:, 0::2], mixed[:, 1::2] = pair.real, pair.imag
        return [rope(s["X1"]), held(rope(s["X2"])), held(mixed)]
    if case["op"] in ("step", "packed"):
        # the recurrence, token by token, all requests and heads at once
        starts, fresh = s["starts"].long(), s["fresh"].long()
        states, Y = s["states"].double(), torch.zeros(s["Y"].shape, dtype=torch.float64, device="cuda")
        C = torch.zeros(len(fresh), *states.shape[1:], dtype=torch.float64, device="cuda")
        old = s["slots_in"] >= 0
        C[old] = states[s["slots_in"][old].long()]
        p1, p2, v, g = (s[x].double() for x in ("P1", "P2", "I", "G"))
        if case["gate"]:
            g = -torch.exp(s["A_log"].double()) * torch.log1p(torch.exp(g + s["dt_bias"].double()))
        S = 1 / (1 + torch.exp(-(p1 * p2).sum(-1) / (TAU * math.sqrt(d))))[..., None]
        q, k = S * p1 / p1.norm(dim=-1, keepdim=True), S * p2 / p2.norm(dim=-1, keepdim=True)
        keep = torch.exp(g)
        order = torch.argsort(fresh, descending=True)  # the longest first: the ones still running come first
        C, first = C[order], starts[:-1][order]
        counts = fresh[order].tolist()
        live = len(counts)
        for t in range(counts[0]):
            while counts[live - 1] <= t:
                live -= 1
            n = first[:live] + t
            now = C[:live]
            now *= keep[n][..., None]
            Y[n] = v[n] + (q[n][..., None] * now).sum(-2)
            now += k[n][..., None] * v[n][..., None, :]
        states[s["slots_out"][order].long()] = C
        return [Y, states]
    if 4.0 * d * case["H"] * sum(f * (c + f) for c, f in _requests(case)) > 4e12:
        return None
    group = case["H"] // case["G"]
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
            k, v = ((x[ids, h] if s["layout"] == 0 else x[ids, :, h]).double() for x in (s["P2_pages"], s["I_pages"]))
            sc = (s["scales"][ids, h] if s["layout"] == 0 else s["scales"][ids, :, h]).double()
            k, v = ((x[..., :d] * sc[..., e, None]).reshape(-1, d)[:c + f] for e, x in enumerate((k, v)))
            for m in range(h * group, (h + 1) * group):
                u = s["P1"][starts[r]:starts[r + 1], m].double() @ k.T / math.sqrt(d)
                w = u / (1 + torch.exp(-u)) - s["lam"] * torch.log((i + 1).double())
                w = torch.where(i == j, 1 / (1 + torch.exp(-u / s["tau_S"])), w)
                w = torch.exp(torch.where(j > i, -math.inf, w) - torch.where(j > i, -math.inf, w).max(1, keepdim=True).values)
                Y[starts[r]:starts[r + 1], m] = (w @ v) / w.sum(1, keepdim=True)
    return [Y]
