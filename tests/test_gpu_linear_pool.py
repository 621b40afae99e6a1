"""Linear Relation over a pool of states on the GPU against the recurrence in 64 bits: packed requests of any lengths,
single tokens, slots of every kind, strong and weak retention, streams, graphs and values that cannot be followed."""
import numpy as np
import pytest
import torch

from linear_pool_cases import TAU, check, inputs, on_gpu, packed
from relation_token_mixing_gb300 import binding as rb

pytestmark = pytest.mark.gpu


def _ok():
    torch.cuda.synchronize()
    assert rb.relation_check_device_status() == 0


@pytest.mark.parametrize("gate", [False, True])
@pytest.mark.parametrize("H,d", [(1, 64), (3, 60), (8, 48), (16, 64)])
def test_single_tokens(H, d, gate):
    x = inputs([1] * 9, H, d, gate, seed=H)
    c = on_gpu(x)
    Y = rb.linear_step(c["P1"], c["P2"], c["I"], c["G"], c["states"], c["slots_in"], c["slots_out"], TAU, c["A_log"],
                       c["dt_bias"])
    _ok()
    assert rb.relation_last_launch_count() == 1
    check(x, Y, c["states"], chunked=False)


@pytest.mark.parametrize("gate", [False, True])
@pytest.mark.parametrize("H,d", [(1, 64), (3, 60), (2, 48), (4, 60)])
def test_few_tokens(H, d, gate):
    x = inputs([0, 1, 2, 5, 16, 15, 3, 0], H, d, gate, seed=7)
    c = on_gpu(x)
    Y = packed(c, max_fresh=16)
    _ok()
    assert rb.relation_last_launch_count() == 1
    check(x, Y, c["states"], chunked=False)


@pytest.mark.parametrize("gate", [False, True])
@pytest.mark.parametrize("H,d", [(1, 64), (3, 60), (2, 48), (4, 60)])
@pytest.mark.parametrize("lengths", [[17], [24], [25], [64], [65, 63], [1, 0, 17, 128, 5, 200, 64, 2], [33, 16, 250, 31, 24, 25]])
def test_requests_of_one_stretch(lengths, H, d, gate):
    x = inputs(lengths, H, d, gate, seed=len(lengths))
    c = on_gpu(x)
    Y = packed(c, max_fresh=max(lengths))
    _ok()
    assert rb.relation_last_launch_count() == (2 if max(lengths) > 16 else 1)  # up to 16 tokens one by one
    check(x, Y, c["states"])


@pytest.mark.parametrize("gate", [False, True])
@pytest.mark.parametrize("H,d", [(2, 64), (3, 60), (1, 48), (2, 60)])
@pytest.mark.parametrize("lengths,bound", [([257], 257), ([1100, 17, 300, 1, 0, 256], 0), ([3, 512, 513, 255, 70], 1000),
                                           ([257], 800), ([770], 770), ([64, 2000, 769, 830, 1], 2000)])
def test_requests_of_many_segments(lengths, bound, H, d, gate):
    x = inputs(lengths, H, d, gate, seed=11)
    c = on_gpu(x)
    Y = packed(c, max_fresh=bound)
    _ok()
    # Cut, if some request may be longer than 640.
    assert rb.relation_last_launch_count() == (4 if min(bound or sum(lengths), sum(lengths)) > 640 else 2)
    check(x, Y, c["states"])


@pytest.mark.parametrize("lengths", [[40, 100, 64], [300, 20, 64], [900, 20, 64]])
@pytest.mark.parametrize("kind", ["strong", "one_channel", "resets", "none", "growing", "lowest", "ragged"])
@pytest.mark.parametrize("d", [64, 60])
def test_retention(kind, lengths, d):
    """Factors that leave the range of a chunk with one reference, retention of nothing and of everything."""
    x = inputs(lengths, 2, d, seed=5)
    N = x["G"].shape[0]
    if kind == "strong":
        x["G"] *= 20.0 / x["G"].abs().mean()
    elif kind == "one_channel":
        x["G"][:, 1, 13] = -9.0
    elif kind == "resets":
        x["G"][::23] = -1e9
    elif kind == "none":
        x["G"].zero_()
    elif kind == "growing":
        x["G"] = 0.002 * torch.rand(x["G"].shape, generator=torch.Generator().manual_seed(1))
    elif kind == "lowest":
        x["G"][N // 2:] = torch.finfo(torch.float32).min
    else:  # strong in some chunks only
        x["G"][: N // 2] *= 40.0
    c = on_gpu(x)
    Y = packed(c, max_fresh=max(lengths))
    _ok()
    check(x, Y, c["states"])


def test_zero_rows_and_large_states():
    x = inputs([70, 4, 20], 2, 60, seed=3)
    x["P1"][3] = 0
    x["P2"][10:30] = 0
    x["I"][40:] *= 1000
    x["states"] *= 50
    c = on_gpu(x)
    Y = packed(c)
    _ok()
    check(x, Y, c["states"])


def test_slots_in_place_shared_and_not_kept():
    """Two requests go on from one slot, one in place, one is new, one's state is not kept, one has no new tokens."""
    x = inputs([20, 3, 70, 1, 0, 0], 2, 64, slots=([0, 0, 2, -1, 5, -1], [1, 4, 2, -1, 3, 6]), seed=9)
    before = x["states"].clone()
    c = on_gpu(x)
    Y = packed(c)
    _ok()
    check(x, Y, c["states"])
    assert torch.equal(c["states"][3].cpu(), before[5]) and (c["states"][6] == 0).all()
    for k in (0, 5):  # read, not written
        assert torch.equal(c["states"][k].cpu(), before[k])


def test_rows_behind_the_last_request_stay():
    x = inputs([30, 2, 18], 3, 60, spare=9, seed=2)
    x["P1"][-9:], x["G"][-9:] = float("nan"), float("nan")
    c = on_gpu(x)
    Y = torch.full_like(c["P1"], 7.0)
    packed(c, Y=Y)
    _ok()
    assert (Y[50:] == 7.0).all()
    for k in ("P1", "G"):
        x[k][-9:] = 0
    check(x, Y, c["states"])


def test_a_request_goes_on_as_if_it_had_never_stopped():
    """A prompt in pieces, from slot to slot, in every split between the kernels."""
    whole = inputs([400], 2, 64, True, slots=([-1], [0]), seed=4)
    cw = on_gpu(whole)
    Yw = packed(cw)
    pool = torch.zeros(2, 2, 64, 64, device="cuda")
    at, ys = 0, []
    for n in (1, 100, 16, 17, 2, 264):
        c = dict(cw, starts=torch.tensor([0, n], dtype=torch.int32, device="cuda"), states=pool)
        for k in ("P1", "P2", "I", "G"):
            c[k] = cw[k][at: at + n].contiguous()
        c["slots_in"] = torch.tensor([-1 if at == 0 else 1], dtype=torch.int32, device="cuda")
        c["slots_out"] = torch.tensor([1], dtype=torch.int32, device="cuda")
        ys.append(packed(c))
        at += n
    _ok()
    check(whole, Yw, cw["states"])
    whole["states"] = torch.zeros(1, 2, 64, 64)
    check(whole, torch.cat(ys), pool[1:])


def test_same_results_from_run_to_run():
    x = on_gpu(inputs([700, 40, 1, 300], 3, 60, True, seed=8))
    first = None
    for _ in range(4):
        pool = x["states"].clone()
        got = packed(dict(x, states=pool)), pool
        if first is None:
            first = got
        assert torch.equal(first[0], got[0]) and torch.equal(first[1], got[1])
    _ok()


@pytest.mark.parametrize("longer", [0, 500])
def test_captured_and_replayed_with_other_lengths(longer):
    lengths = [[300 + longer, 17, 1], [5, 290 + longer, 23], [0, 16, 302 + longer]]
    xs = [inputs(n, 2, 64, slots=([0, 1, 2], [0, 1, 2]), seed=20 + k) for k, n in enumerate(lengths)]
    c = on_gpu(xs[0])
    Y = torch.empty_like(c["P1"])
    ws = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
    packed(c, max_fresh=310 + longer, Y=Y, workspace=ws)  # loads the kernels
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        packed(c, max_fresh=310 + longer, Y=Y, workspace=ws)
    for x in xs:
        for k, t in x.items():
            if t is not None:
                c[k].copy_(t)
        graph.replay()
        _ok()
        check(x, Y, c["states"])


def test_two_captured_graphs_over_one_workspace():
    xs = [inputs([900, 3, 70], 2, 64, seed=30), inputs([20, 700, 800, 1], 2, 64, True, seed=31)]
    cs = [on_gpu(x) for x in xs]
    ws = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
    ys, graphs = [torch.empty_like(c["P1"]) for c in cs], []
    for c, Y in zip(cs, ys):
        packed(c, Y=Y, workspace=ws)  # loads the kernels
        torch.cuda.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            packed(c, Y=Y, workspace=ws)
    for k in (0, 1, 1, 0):
        cs[k]["states"].copy_(xs[k]["states"])
        ys[k].zero_()
        graphs[k].replay()
    _ok()
    for x, c, Y in zip(xs, cs, ys):
        check(x, Y, c["states"])


@pytest.mark.parametrize("lengths", [[90, 130, 5, 40], [90, 900, 5, 40]])
@pytest.mark.parametrize("which", ["P1", "P2", "I", "G"])
def test_a_value_that_is_not_finite_stays_with_its_head(which, lengths):
    """NaN in one head of one token: that head from that token on, at most 63 rows before it, and its state; no other."""
    x = inputs(lengths, 2, 64, seed=16)
    c = on_gpu(x)
    at = lengths[0] + 100
    c[which][at, 1, 5] = float("nan")
    Y = packed(c)
    _ok()
    end = lengths[0] + lengths[1]
    assert torch.isnan(Y[at: end, 1].float()).any(-1).all()
    assert torch.isnan(c["states"][int(c["slots_out"][1]), 1]).any()
    # The rest as if it had not been.
    want, pool = packed(dict(on_gpu(x), states=(clean := x["states"].cuda()))), clean
    keep = torch.ones(Y.shape[:2], dtype=torch.bool, device="cuda")
    keep[at - 63: end, 1] = False
    assert torch.equal(Y[keep], want[keep])
    mine = torch.ones(pool.shape[:2], dtype=torch.bool, device="cuda")
    mine[int(c["slots_out"][1]), 1] = False
    assert torch.equal(c["states"][mine], pool[mine])
    check(x, want, pool)


@pytest.mark.parametrize("longest", [300, 900])
def test_on_another_stream(longest):
    x = inputs([longest, 2, 40], 2, 64, seed=6)
    c = on_gpu(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    Y = packed(c, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    _ok()
    check(x, Y, c["states"])


@pytest.mark.parametrize("longest", [280, 900])
def test_calls_in_flight_over_one_workspace(longest):
    """Steps queued one after another, each going on from the state of the one before."""
    x = inputs([longest, 30, 1], 2, 64, slots=([0, 1, 2], [0, 1, 2]), seed=12)
    c = on_gpu(x)
    ws = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
    ys = [packed(c, workspace=ws) for _ in range(5)]
    _ok()
    for Y in ys:  # the same steps one at a time
        alone = on_gpu(x)
        assert torch.equal(packed(alone), Y)
        check(x, Y, alone["states"])
        x["states"] = alone["states"].cpu()
    assert torch.equal(x["states"], c["states"].cpu())


@pytest.mark.parametrize("what", ["past", "descending", "bound", "slot_in", "slot_out"])
def test_values_that_cannot_be_followed_are_reported(what):
    x = inputs([20, 3, 40], 2, 64, slots=([0, 1, 2], [3, 4, 5]), seed=13)
    before = x["states"].clone()
    c = on_gpu(x)
    if what == "past":
        c["starts"][3] = 64
    elif what == "descending":
        c["starts"][1], c["starts"][2] = 23, 20
    elif what == "slot_in":
        c["slots_in"][1] = 6
    elif what == "slot_out":
        c["slots_out"][1] = 1 << 30
    Y = torch.full_like(c["P1"], 7.0)
    packed(c, max_fresh=30 if what == "bound" else 0, Y=Y)
    torch.cuda.synchronize()
    assert rb.relation_check_device_status() == 1 and rb.relation_check_device_status() == 0
    states = c["states"].cpu()
    if what in ("past", "bound"):  # the third request is skipped, the others are not
        assert (Y[23:] == 7.0).all() and torch.equal(states[5], before[5]) and not torch.equal(states[3], before[3])
    elif what == "descending":
        assert torch.equal(states[4], before[4])
    elif what == "slot_in":  # as a new request
        x["slots_in"][1] = -1
        check(x, Y, c["states"])
    else:
        x["slots_out"][1] = -1
        check(x, Y, c["states"])


def test_more_requests_than_a_block_has_threads():
    lengths = [(7 * r) % 40 if r % 50 else 300 for r in range(400)]
    x = inputs(lengths, 1, 48, slots=(list(range(400)), list(range(400))), seed=14)
    c = on_gpu(x)
    Y = packed(c)
    _ok()
    check(x, Y, c["states"])


def test_no_new_tokens_at_all():
    x = inputs([0, 0], 2, 64, slots=([0, -1], [2, 1]), seed=15)
    before = x["states"].clone()
    c = on_gpu(x)
    Y = packed(c)
    _ok()
    assert Y.shape[0] == 0
    assert torch.equal(c["states"][2].cpu(), before[0]) and (c["states"][1] == 0).all()


def test_agrees_with_the_dense_forward():
    B, H, T, d = 2, 3, 333, 60
    x = inputs([T] * B, H, d, slots=([-1] * B, list(range(B))), seed=16)
    c = on_gpu(x)
    Y = packed(c)
    dense = {k: c[k].view(B, T, H, d) for k in ("P1", "P2", "I", "G")}
    Yd, state = rb.linear_fwd(dense["P1"], dense["P2"], dense["I"], dense["G"], TAU, rb.RELATION_LAYOUT_BTHD, True)
    _ok()
    check(x, Y, c["states"])
    scale = float(Yd.float().abs().max())
    assert float((Y.view(B, T, H, d).float() - Yd.float()).abs().max()) <= 2e-2 * scale  # both within 1e-2
    assert float((c["states"] - state).abs().max()) <= 2e-2 * float(np.abs(state.cpu().numpy()).max())


def test_slots_past_32_bits():
    """A pool of more than 2^32 floats: its last slots against the same states in a small pool."""
    H, d, slots = 8, 64, 132000
    big = rb.linear_states(slots, H, d)
    assert big.numel() > 1 << 32
    x = inputs([70, 1, 5, 900], H, d, slots=([4, 5, -1, 6], [0, 5, 1, 2]), seed=17)
    small = on_gpu(x)
    n = small["states"].shape[0]
    big[-n:] = small["states"]
    Y = packed(small)
    up = lambda s: torch.where(s < 0, s, s + slots - n)  # noqa: E731
    Yb = packed(dict(small, states=big, slots_in=up(small["slots_in"]), slots_out=up(small["slots_out"])))
    _ok()
    assert torch.equal(Y, Yb) and torch.equal(big[-n:], small["states"])
    assert (big[:-n] == 0).all()


@pytest.mark.parametrize("max_fresh", [0, 1])
def test_rows_past_32_bits(max_fresh):
    """Packed tensors of more than 2^31 values: the last request's heads against a call of their own."""
    H, d = 1024, 64
    lengths = [33000, 17, 1] if max_fresh == 0 else [1] * 33018
    N, gen = sum(lengths), torch.Generator("cuda").manual_seed(18)
    assert N * H * d > 1 << 31
    P1, P2, I = (torch.randn(N, H, d, generator=gen, device="cuda", dtype=torch.bfloat16) for _ in range(3))
    G = -0.1 * torch.rand(N, H, d, generator=gen, device="cuda")
    starts = torch.tensor([0] + lengths, device="cuda").cumsum(0).int()
    R, last = len(lengths), 3
    keep = torch.full((R,), -1, dtype=torch.int32, device="cuda")
    keep[-last:] = torch.arange(last, device="cuda", dtype=torch.int32)
    states = rb.linear_states(last, H, d)
    Y = rb.linear_packed_fwd(P1, P2, I, G, starts, states, torch.full_like(keep, -1), keep, max_fresh, TAU)
    _ok()
    n = sum(lengths[-2:])  # the last two requests, first and last head
    for h in (0, H - 1):
        x = dict(P1=P1, P2=P2, I=I, G=G)
        x = {k: t[-n:, h: h + 1].contiguous().cpu() for k, t in x.items()}
        x |= dict(A_log=None, dt_bias=None, starts=torch.tensor([0, lengths[-2], n]), states=torch.zeros(2, 1, d, d),
                  slots_in=torch.tensor([-1, -1]), slots_out=torch.tensor([0, 1]))
        check(x, Y[-n:, h: h + 1].cpu(), states[-2:, h: h + 1].cpu())
