"""Host model of the roles of the paged tensor-core forward over 8-bit pages (no GPU): as the model for bf16 pages, with
the rings of whole numbers that the copies fill and the four warps that make bf16 tiles of them.

The converting warps take the tiles in the order K0, K1, V0, K2, V1, ... of the block's whole stretch, with one loop for
both; a tile is full when all four have written their rows, its ring's place empty when all four have read it.  No turns and
no cleared tiles here: the softmax goes in blocks of columns, and keys past the end are written as zeros."""
import os
import random
import re

import pytest

from test_paged_roles import CASES, CSRC, SLOTS, Alias, Bar, pieces


def run(work, wide, seed, overwrite=False):
    """One worker's roles over its pieces; raises Alias, returns whether all roles ended.  overwrite: a mistake,
    tiles written without waiting for their place."""
    rnd = random.Random(seed)
    stages, qbufs = (2, 1) if wide else (4, 2)
    v_stages = ring = stages // 2
    bars = lambda n, count: [Bar(count) for _ in range(n)]  # noqa: E731
    piece_full, piece_free = bars(SLOTS, 1), bars(SLOTS, 15)
    q_full, q_free = bars(2, 4 if wide else 1), bars(2, 1)
    k_full, k_empty, v_full, v_empty = bars(stages, 4), bars(stages, 1), bars(v_stages, 4), bars(v_stages, 1)
    k8_full, v8_full, k8_empty, v8_empty = bars(ring, 1), bars(ring, 1), bars(ring, 4), bars(ring, 4)
    s_full, o_done, s_free, p_full = bars(2, 1), bars(2, 1), bars(2, 4), bars(2, 4)  # a warp's 32 arrivals as one
    line = [(steps, most) for steps, most, _ in work] + [((0, 0), -1)]

    def take(seg):
        yield piece_full[seg % SLOTS], seg // SLOTS

    def give(seg):
        piece_free[seg % SLOTS].arrive()

    def load(x, most, full, empty):
        for y in range(x, x + most):
            if y >= ring:
                yield empty[y % ring], y // ring - 1
            full[y % ring].arrive()
            yield None

    def walker():
        x = 0
        for seg, (_, most) in enumerate(line):
            if seg >= SLOTS:
                yield piece_free[seg % SLOTS], seg // SLOTS - 1
            piece_full[seg % SLOTS].arrive()
            if most < 0:
                return
            yield from load(x, most, k8_full, k8_empty)
            x += most

    def values():
        x = 0
        for seg, (_, most) in enumerate(line):
            yield from take(seg)
            give(seg)
            if most < 0:
                return
            yield from load(x, most, v8_full, v8_empty)
            x += most

    def converter():
        seg = left = 0

        def next_tile():  # whether there is one; its piece is taken and given back at once
            nonlocal seg, left
            if left == 0:
                yield from take(seg)
                left = line[seg][1]
                give(seg)
                seg += 1
                if left < 0:
                    return False
            left -= 1
            return True

        def item(which, y):
            n = v_stages if which else stages
            yield (v8_full if which else k8_full)[y % ring], y // ring
            if y >= n and not overwrite:
                yield (v_empty if which else k_empty)[y % n], y // n - 1
            yield None
            (v8_empty if which else k8_empty)[y % ring].arrive()
            (v_full if which else k_full)[y % n].arrive()

        more = yield from next_tile()
        z = 0
        ended = not more
        while True:
            which = z > 0 and z % 2 == 0
            y = z // 2 - 1 if which else (z + 1) // 2
            if not which:
                if not more:
                    if z == 0:
                        return
                    ended = True
                    z += 1
                    continue
                more = yield from next_tile()
            yield from item(which, y)
            if which and ended:
                return
            z += 1

    def queries():
        for seg, (_, most) in enumerate(line):
            yield from take(seg)
            give(seg)
            if most < 0:
                return
            if not wide:
                if seg >= qbufs:
                    yield q_free[seg % qbufs], seg // qbufs - 1
                q_full[seg % qbufs].arrive()
            yield None

    def softmax(t):
        def next_q(seg):
            if wide:
                yield from take(seg)
                if line[seg][0][t] > 0:
                    q_full[t].arrive()

        n = 0
        yield from next_q(0)
        for seg, (steps, most) in enumerate(line):
            yield from take(seg)
            if most < 0:
                return
            for j in range(steps[t]):
                yield s_full[t], n + j
                if j > 0 and (not wide or rnd.random() < .5):
                    yield o_done[t], n + j - 1
                if not wide:
                    s_free[t].arrive()
                p_full[t].arrive()
                yield None
            yield from next_q(seg + 1)
            if steps[t]:
                yield o_done[t], n + steps[t] - 1
            n += steps[t]
            give(seg)

    def products():
        k, st, begun, halves = 0, [0, 0], [False, False], [0, 0]

        def read(seg):
            yield from take(seg)
            give(seg)
            return line[seg]

        def q_wait(seg, t):
            if not wide:
                yield q_full[seg % qbufs], seg // qbufs
            else:
                yield q_full[t], halves[t]
                halves[t] += 1

        now, seg = (yield from read(0)), 0
        while now[1] >= 0:
            steps, most = now
            yield k_full[k % stages], k // stages
            for t in (0, 1):
                if steps[t] and not begun[t]:
                    yield from q_wait(seg, t)
                    if not wide and st[t]:
                        yield s_free[t], st[t] - 1
                    s_full[t].arrive()
                begun[t] = False
            k_empty[k % stages].arrive()
            if not wide and most == 1:
                q_free[seg % qbufs].arrive()
            after = None
            for j in range(most):
                ready = False
                for t in (0, 1):
                    if j >= steps[t]:
                        continue
                    if not wide:
                        yield s_free[t], st[t] + j
                        if j + 1 < steps[t]:
                            yield k_full[(k + j + 1) % stages], (k + j + 1) // stages
                            s_full[t].arrive()
                        else:
                            if after is None:
                                after = yield from read(seg + 1)
                            if after[0][t]:
                                yield from q_wait(seg + 1, t)
                                yield k_full[(k + most) % stages], (k + most) // stages
                                s_full[t].arrive()
                                begun[t] = True
                    yield p_full[t], st[t] + j
                    if not ready:
                        ready = True
                        yield v_full[(k + j) % v_stages], (k + j) // v_stages
                    o_done[t].arrive()
                    if wide and j + 1 < steps[t]:
                        yield k_full[(k + j + 1) % stages], (k + j + 1) // stages
                        s_full[t].arrive()
                if j + 1 < most:
                    k_empty[(k + j + 1) % stages].arrive()
                if not wide and j + 2 == most:
                    q_free[seg % qbufs].arrive()
                v_empty[(k + j) % v_stages].arrive()
                yield None
            if after is None:
                after = yield from read(seg + 1)
            k, st = k + most, [st[t] + steps[t] for t in (0, 1)]
            now, seg = after, seg + 1

    roles = [walker(), values(), queries(), products()] + [converter() for _ in range(4)] + \
        [softmax(t) for t in (0, 1) for _ in range(4)]
    alive = [[r, None] for r in roles]
    while alive:
        moved = False
        rnd.shuffle(alive)
        for role in list(alive):
            if role[1] is not None and not role[1][0].done(role[1][1]):
                continue
            moved = True
            try:
                role[1] = next(role[0])
            except StopIteration:
                alive.remove(role)
        if not moved:
            return False
    return True


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_roles_end_and_no_wait_is_two_phases_away(case, wide):
    for worker, work in enumerate(pieces(*CASES[case])):
        for seed in range(3):
            assert run(work, wide, 100 * worker + seed)


def _caught(wide, **mistake):
    for case in CASES:
        for worker, work in enumerate(pieces(*case)):
            for seed in range(3):
                try:
                    if not run(work, wide, 100 * worker + seed, **mistake):
                        return True
                except Alias:
                    return True
    return False


def test_a_planted_mistake_is_caught():
    assert _caught(False, overwrite=True) and _caught(True, overwrite=True)


def test_the_model_follows_the_kernel():
    text = re.sub(r"\s+", " ", open(os.path.join(CSRC, "paged_tc.cu")).read())
    for piece in (
            "kVStages = Q8 ? kStages / 2 : kStages;", "kRing = Q8 ? kStages / 2 : kStages;",
            "mbar_init(&bars->piece_free[x], 15)", "mbar_init(&bars->k_full[s], Q8 ? 4 : 1)",
            "mbar_init(&bars->v_full[s], Q8 ? 4 : 1)", "mbar_init(&bars->k8_empty[s], 4)",
            "mbar_init(&bars->v8_empty[s], 4)", "if (Q8) pc.tail = -1;",
            "const int which = z > 0 && (z & 1) == 0, y = which ? z / 2 - 1 : (z + 1) / 2;",
            "mbar_wait_warp(&full8[from], (y / C::kRing) & 1, abort_flag, v.status, kDevTimeoutFull)",
            "(y >= stages && !ptx::mbar_wait_warp(&empty[to], (y / stages - 1) & 1,",
            "n_pair = C::kSepP || Q8 ? 0 : min(pc->steps[0], pc->steps[1]);",
            "wait(&bars->v_full[s], (kt + j) / C::kVStages, kDevTimeoutFull)"):
        assert piece in text, piece
