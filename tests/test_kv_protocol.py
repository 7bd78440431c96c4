"""Barrier protocol of the tiled attention kernel, on the CPU.

An event-driven model of the roles of `tiled_kernel` (csrc/w4kv_attn_tiled.cu)
for one block: the two softmax groups, the two MMA warps, the widening warps
and the scales' warp, each a generator that yields what it waits for, and the
mbarriers with the one-bit parity of the hardware: a waiter that a barrier
passes twice waits for good.  Schedules are random and adversarial (one role
is only run when no other can move).  A segment is (steps, steps that stream A
takes part in, split): split segments hold one row tile whose steps the streams
take in turn.
"""
import random

import pytest

BUFFERS, SCALE_STAGES = 3, 4
ROLES = ("softmax 0", "softmax 1", "mma 0", "mma 1", "widen", "scales")


class Bar:
    """mbarrier: `count` arrivals complete a phase; a wait on parity p passes
    while the phase under way has the other parity."""

    def __init__(self, count):
        self.count = self.pending = count
        self.phase = 0

    def arrive(self):
        self.pending -= 1
        if self.pending == 0:
            self.phase += 1
            self.pending = self.count

    def passed(self, parity):
        return (self.phase & 1) != parity


def own_steps(seg, t):
    """Steps in which stream t has MMAs of its own."""
    ns, first, split = seg
    if split:
        return (ns + 1 - t) // 2
    return first if t == 0 else ns


def run_block(segments, schedule, skip=True):
    """Runs the roles to the end; None, or the roles that wait for good.
    `skip`: a stream passes q_full only in segments with steps of its own."""
    q_full = [Bar(1) for _ in range(2)]
    s_full = [Bar(1) for _ in range(2)]
    p_full = [Bar(1) for _ in range(2)]
    pv_done = [Bar(1) for _ in range(2)]
    full = [Bar(1) for _ in range(BUFFERS)]
    empty = [Bar(2) for _ in range(BUFFERS)]
    sc_full = [Bar(1) for _ in range(SCALE_STAGES)]
    sc_empty = [Bar(2) for _ in range(SCALE_STAGES)]
    joined = Bar(2)
    q_of = [None, None]  # segment whose queries lie in the stream's tile

    def softmax(t):
        step = own_no = joins = 0
        for k, seg in enumerate(segments):
            ns, first, split = seg
            own = own_steps(seg, t)
            if own or not skip:
                q_of[t] = k
                q_full[t].arrive()
                yield None
            for j in range(ns):
                yield sc_full[step % SCALE_STAGES], (step // SCALE_STAGES) & 1
                if (j & 1) == t if split else j < own:
                    yield s_full[t], own_no & 1
                    p_full[t].arrive()
                    yield None
                    own_no += 1
                sc_empty[step % SCALE_STAGES].arrive()
                yield None
                step += 1
            if own:
                yield pv_done[t], (own_no - 1) & 1
            if split:
                for _ in range(3):
                    joined.arrive()
                    yield None
                    yield joined, joins & 1
                    joins += 1

    def mma(t):
        step0 = n_p = n_q = 0

        def filled(n):
            return full[n % BUFFERS], (n // BUFFERS) & 1

        for k, seg in enumerate(segments):
            ns, first, split = seg
            own = own_steps(seg, t)
            if own or not skip:
                yield q_full[t], n_q & 1
                n_q += 1

            def score(n):
                assert q_of[t] == k, "queries of another segment"
                s_full[t].arrive()
                empty[n % BUFFERS].arrive()

            def output(n):
                pv_done[t].arrive()
                empty[n % BUFFERS].arrive()

            if split:
                for j in range(ns):
                    n = 2 * (step0 + j)
                    yield filled(n)
                    if (j & 1) == t:
                        score(n)
                    else:
                        empty[n % BUFFERS].arrive()
                    yield None
                    yield filled(n + 1)
                    if (j & 1) == t:
                        yield p_full[t], n_p & 1
                        n_p += 1
                        output(n + 1)
                    else:
                        empty[(n + 1) % BUFFERS].arrive()
                    yield None
            else:
                if own:
                    yield filled(2 * step0)
                    score(2 * step0)
                    yield None
                for j in range(own):
                    n = 2 * (step0 + j) + 1
                    yield filled(n)
                    if j + 1 < own:
                        yield filled(n + 1)
                    yield p_full[t], n_p & 1
                    n_p += 1
                    output(n)
                    if j + 1 < own:
                        score(n + 1)
                    yield None
                for j in range(own, ns):
                    for i in range(2):
                        yield filled(2 * (step0 + j) + i)
                        empty[(2 * (step0 + j) + i) % BUFFERS].arrive()
                        yield None
            step0 += ns

    def widen():
        for n in range(2 * sum(s[0] for s in segments)):
            yield empty[n % BUFFERS], ((n // BUFFERS) & 1) ^ 1
            full[n % BUFFERS].arrive()
            yield None

    def scales():
        for n in range(sum(s[0] for s in segments)):
            yield sc_empty[n % SCALE_STAGES], ((n // SCALE_STAGES) & 1) ^ 1
            sc_full[n % SCALE_STAGES].arrive()
            yield None

    roles = dict(zip(ROLES, (softmax(0), softmax(1), mma(0), mma(1), widen(), scales())))
    waits = dict.fromkeys(roles)
    while roles:
        ready = [r for r in roles if waits[r] is None or waits[r][0].passed(waits[r][1])]
        if not ready:
            return sorted(roles)
        r = schedule(ready)
        try:
            waits[r] = next(roles[r])
        except StopIteration:
            del roles[r]
    return None


def schedules(seed):
    """Random choice, and each role in turn run only when no other can move,
    or before all others."""
    rng = random.Random(seed)
    yield rng.choice
    for role in ROLES:
        yield lambda ready, role=role: rng.choice([r for r in ready if r != role] or ready)
        yield lambda ready, role=role: role if role in ready else rng.choice(ready)


# Rows of a padded batch (kv_lens = 0) see nothing: one step, none of stream A's.
NOTHING = (1, 0, False)
ITEMS = {
    "rows that see nothing": [NOTHING] * 12,
    "among chunks": [(5, 4, False), NOTHING, NOTHING, NOTHING, (9, 9, False), NOTHING, NOTHING, NOTHING],
    "split, one step each": [(1, 1, True)] * 12,
    "all kinds": [(1, 1, True), NOTHING, (2, 2, True), NOTHING, NOTHING, (3, 1, False), (1, 0, False),
                  (1, 1, True), (1, 1, True), (4, 0, False), (7, 7, True), NOTHING],
}


@pytest.mark.parametrize("name", ITEMS)
def test_no_deadlock(name):
    for seed in range(20):
        for schedule in schedules(seed):
            assert run_block(ITEMS[name], schedule) is None


@pytest.mark.parametrize("seed", range(40))
def test_no_deadlock_random_segments(seed):
    rng = random.Random(seed)
    segments = []
    for _ in range(rng.randint(1, 14)):
        ns = rng.choice((1, 1, 1, 2, 3, 6))
        split = rng.random() < 0.4
        segments.append((ns, ns if split else rng.choice((0, 0, ns, max(0, ns - 1))), split))
    for schedule in schedules(seed):
        assert run_block(segments, schedule) is None, segments


def test_model_finds_the_double_pass():
    """The model is not vacuous: with queries announced in every segment, stream
    A's softmax can pass q_full twice before its MMA warp has looked, and the
    block stops."""
    stuck = [run_block(ITEMS["rows that see nothing"], s, skip=False)
             for seed in range(20) for s in schedules(seed)]
    assert any(s is not None and "mma 0" in s for s in stuck)
