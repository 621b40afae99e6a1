"""Host model of the roles of the paged tensor-core forward (no GPU).

The kernel's warps hand work on through mbarriers: the walker's pieces and P2 tiles, the I~ tiles (with the keys past a
request's end cleared), the queries, the scores, the weights, the outputs and, at d > 64, the turns of the halves'
softmax warps.  An mbarrier wait by parity tells a phase from the next only: it is sound only if the barrier is, whenever
the wait is made, in the awaited phase or done with it and in the next.  The model runs every role as a coroutine over
pieces of random requests, in random orders, and checks that

- every role ends (no wait is left unsatisfied);
- no wait is ever made two phases away from its barrier (the parity would lie);
- no arrival is one too many for its phase.

Two planted mistakes, both once made, have to be caught: the queries of a half without steps counted as a phase, and
the tile that a request ends inside awaited long before it is loaded.  The last test holds the counts and the order of
the products to the kernel's source.
"""
import os
import random
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "relation_token_mixing_gb300", "csrc")
KEYS, ROWS, BM, EXTRA, SLOTS, MIN_TILES = 128, 256, 128, 2, 4, 4


class Alias(Exception):
    pass


class Bar:
    def __init__(self, count):
        self.count = self.left = count
        self.phase = 0

    def arrive(self):
        self.left -= 1
        assert self.left >= 0
        if self.left == 0:
            self.phase, self.left = self.phase + 1, self.count

    def done(self, phase):
        if phase not in (self.phase, self.phase - 1):
            raise Alias((phase, self.phase))
        return phase < self.phase


def pieces(requests, group, heads, workers):
    """Each worker's pieces: (steps of the two halves, their maximum, tile the request ends inside or -1)."""
    units, at = [], 0
    for c, fresh in requests:
        rows = fresh * group
        for _ in range(heads):
            for q in range(-(-rows // ROWS)):
                n = (c + (min(rows, (q + 1) * ROWS) - 1) // group + KEYS) // KEYS
                units.append((at + EXTRA, n, c, rows, q))
                at += EXTRA + n
    used = max(1, min(workers, at // MIN_TILES))
    each, extra = at // used, at % used
    out = []
    for w in range(workers):
        lo, hi = (each * x + min(x, extra) for x in (min(w, used), min(w + 1, used)))
        mine = []
        for u0, n, c, rows, q in units:
            j0, j1 = max(0, lo - u0), min(n, hi - u0)
            if j0 >= j1:
                continue
            steps = []
            for t in (0, 1):
                here = max(0, min(BM, rows - q * ROWS - t * BM))
                seen = (c + (q * ROWS + t * BM + here - 1) // group + KEYS) // KEYS if here else 0
                steps.append(max(0, min(j1, seen) - j0))
            most, end = max(steps), c + rows // group
            inside = end % KEYS != 0 and j0 <= end // KEYS < j0 + most
            mine.append((tuple(steps), most, end // KEYS - j0 if inside else -1))
        out.append(mine)
    return out


def run(work, wide, seed, count_idle_queries=False, early_tail=False):
    """One worker's roles over its pieces; raises Alias, returns whether all roles ended."""
    rnd = random.Random(seed)
    stages, qbufs = (2, 1) if wide else (4, 2)
    bars = lambda n, count: [Bar(count) for _ in range(n)]  # noqa: E731
    piece_full, piece_free = bars(SLOTS, 1), bars(SLOTS, 11)
    q_full, q_free = bars(2, 4 if wide else 1), bars(2, 1)
    k_full, k_empty, v_full, v_empty = (bars(stages, 1) for _ in range(4))
    v_clean = bars(4, 1)
    s_full, o_done, s_free, p_full = bars(2, 1), bars(2, 1), bars(2, 4), bars(2, 4)  # a warp's 32 arrivals as one
    turn = [bars(4, 1) for _ in range(2)]
    line = list(work) + [((0, 0), -1, -1)]

    def take(seg):
        yield piece_full[seg % SLOTS], seg // SLOTS

    def give(seg):
        piece_free[seg % SLOTS].arrive()

    def walker():
        x = 0
        for seg, (_, most, _) in enumerate(line):
            if seg >= SLOTS:
                yield piece_free[seg % SLOTS], seg // SLOTS - 1
            piece_full[seg % SLOTS].arrive()
            for _ in range(most):
                if x >= stages:
                    yield k_empty[x % stages], x // stages - 1
                k_full[x % stages].arrive()
                x += 1
                yield None

    def values():
        x = tails = 0
        for seg, (_, most, tail) in enumerate(line):
            yield from take(seg)
            give(seg)
            if most < 0:
                return
            if early_tail and tail >= 0:
                yield v_full[(x + tail) % stages], (x + tail) // stages
            for _ in range(most):
                if x >= stages:
                    yield v_empty[x % stages], x // stages - 1
                v_full[x % stages].arrive()
                x += 1
                yield None
            if tail >= 0:
                assert tail == most - 1
                yield v_full[(x - 1) % stages], (x - 1) // stages
                v_clean[tails % 4].arrive()
                tails += 1

    def queries():
        for seg, (_, most, _) in enumerate(line):
            yield from take(seg)
            give(seg)
            if most < 0:
                return
            if not wide:
                if seg >= qbufs:
                    yield q_free[seg % qbufs], seg // qbufs - 1
                q_full[seg % qbufs].arrive()
            yield None

    def softmax(t, quarter):
        def next_q(seg):
            if wide:
                yield from take(seg)
                if line[seg][0][t] > 0 or (count_idle_queries and line[seg][1] >= 0):
                    q_full[t].arrive()

        n = pairs = 0
        yield from next_q(0)
        for seg, (steps, most, _) in enumerate(line):
            yield from take(seg)
            if most < 0:
                return
            paired = min(steps) if wide else 0
            for j in range(steps[t]):
                yield s_full[t], n + j
                if not wide:
                    if j > 0:
                        yield o_done[t], n + j - 1
                    s_free[t].arrive()
                else:
                    x = pairs + j
                    if j < paired and x + t > 0:
                        yield turn[t][quarter], x + t - 1
                    yield None
                    if j < paired:
                        turn[t ^ 1][quarter].arrive()
                    if j > 0 and rnd.random() < .2:  # the maximum rose
                        yield o_done[t], n + j - 1
                p_full[t].arrive()
                yield None
            yield from next_q(seg + 1)
            if steps[t]:
                yield o_done[t], n + steps[t] - 1
            n, pairs = n + steps[t], pairs + paired
            give(seg)

    def products():
        k = tails = 0
        st, begun, halves = [0, 0], [False, False], [0, 0]

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
            steps, most, tail = now
            yield k_full[k % stages], k // stages
            for t in (0, 1):
                if count_idle_queries and steps[t] == 0 and wide:
                    yield from q_wait(seg, t)
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
                        if j == tail:
                            yield v_clean[tails % 4], tails // 4
                        else:
                            yield v_full[(k + j) % stages], (k + j) // stages
                    o_done[t].arrive()
                    if wide and j + 1 < steps[t]:
                        yield k_full[(k + j + 1) % stages], (k + j + 1) // stages
                        s_full[t].arrive()
                if j + 1 < most:
                    k_empty[(k + j + 1) % stages].arrive()
                if not wide and j + 2 == most:
                    q_free[seg % qbufs].arrive()
                v_empty[(k + j) % stages].arrive()
                yield None
            if after is None:
                after = yield from read(seg + 1)
            k, tails = k + most, tails + (tail >= 0)
            st = [st[t] + steps[t] for t in (0, 1)]
            now, seg = after, seg + 1

    alive = [[r, None] for r in [walker(), values(), queries(), products()] +
             [softmax(t, w) for t in (0, 1) for w in range(4)]]
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


CASES = [  # requests (cached, new tokens), heads of a group, cache heads, workers
    ([(0, 512), (0, 567), (0, 53), (0, 379)], 1, 3, 11),
    ([(100, 40), (3000, 130), (0, 129), (127, 129)], 2, 4, 7),
    ([(9000, 300)], 4, 2, 9),
    ([(1, 20), (130, 18), (255, 33), (0, 17), (640, 64)], 1, 2, 3),
    ([(5000, 17), (64, 25), (127, 17)], 8, 1, 5),
]


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


def test_planted_mistakes_are_caught():
    assert _caught(True, count_idle_queries=True)
    assert _caught(False, early_tail=True)


def test_the_model_follows_the_kernel():
    text = re.sub(r"\s+", " ", open(os.path.join(CSRC, "paged_tc.cu")).read())
    for piece in (
            "kBM = 128, kRows = 256, kKeys = 128;", "kStages = D == 64 ? 4 : 2;", "kQBufs = D == 64 ? 2 : 1;",
            "using TcTiling = Tiling<kRows, kKeys, 2>;", "constexpr int kMinTiles = 4;", "constexpr int kSlots = 4;",
            "mbar_init(&bars->piece_free[x], 11)", "mbar_init(&bars->q_full[t], C::kSepP ? 1 : 4)",
            "mbar_init(&bars->s_free[t], 128)", "mbar_init(&bars->p_full[t], 128)",
            "wait(&bars->q_full[t], halves[t]++, kDevTimeoutFull)",
            "if (sg.steps[t] == 0 || begun[t]) continue; if (!q_wait(seg, t)) break;",
            "if (pc != nullptr && pc->steps[t] > 0) load_q(",
            "v_ready = j == sg.tail ? wait(&bars->v_clean[tails % 4], tails / 4, kDevTimeoutFull)",
            "if (C::kSepP && sg.most == 1) ptx::mma_commit_elect(&bars->q_free[qb]);",
            "if (!ptx::mbar_wait_warp(&bars->v_full[s], ((x - 1) / C::kStages) & 1, abort_flag, v.status,"):
        assert piece in text, piece
