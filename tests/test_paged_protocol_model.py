"""CPU model of the paged kernel's barrier protocol (attn_paged_kernel.cuh; no
GPU), with waits that run out.

* The producer, unit by unit: waits for Q's slot (uempty), arms ufull with Q's
  load, then per tile waits for the stage (empty), arms it (full) with its
  loads.  At the end it hands over the end of the line, on ufull without a load.
  A wait that runs out ends it.  Either way it first settles: waits, up to twice the limit,
  for the last load of every stage, and for Q's unless the end was handed over
  (ufull is two phases on by then).
* Consumer warps, in groups of four: wait for ufull, meet (a warp whose wait ran
  out ends its group here), read Q, arrive on uempty; per tile wait for full,
  read, arrive on empty.  A warp whose wait ran out goes on to the meeting
  point without reading or arriving.
* Loads land after random delays; in some runs one of them takes longer than a
  wait's limit.

Checked: every role ends; no load is in flight when the last one does; no
barrier is armed in a phase that has not completed, nor seen two phases ahead; a
slot is rewritten only when every warp has read it; without slow loads no wait
runs out and every warp reads every tile."""

import random

import pytest

LIMIT = 400  # ticks


class Barrier:
    def __init__(self, count):
        self.count, self.pending, self.loads, self.phase = count, count, 0, 0

    def _turn(self):
        if self.pending == 0 and self.loads == 0:
            self.pending, self.phase = self.count, self.phase + 1

    def arrive(self, loads=0):
        assert self.pending > 0, "armed in a phase that has not completed"
        self.pending, self.loads = self.pending - 1, self.loads + loads
        self._turn()

    def land(self):
        self.loads -= 1
        self._turn()

    def parity_done(self, parity):
        """What the kernel's parity wait sees."""
        return (self.phase & 1) != parity


def run(units, stages, groups, seed, slow=None, mistake=None):
    """units: tiles of each; slow: the index of the load that takes long (counted
    as issued).  Returns (waits that ran out, tiles read by every warp)."""
    rng = random.Random(seed)
    warps = 4 * groups
    full, empty = [Barrier(1) for _ in range(stages)], [Barrier(warps) for _ in range(stages)]
    ufull, uempty = Barrier(1), Barrier(warps)
    now, ran_out, flying, issued = [0], [0], [], [0]
    slots, readers = [None] * stages, [set() for _ in range(stages)]
    unit_now, read = [None], [[] for _ in range(warps)]

    def load(bar):
        delay = int(1.5 * LIMIT) if issued[0] == slow else rng.randint(1, 20)
        issued[0] += 1
        flying.append((now[0] + delay, bar))

    def wait(bar, parity, settling=False):
        """True once the phase of this parity has completed, False after LIMIT."""
        start = now[0]
        while not bar.parity_done(parity):
            if now[0] - start > (2 * LIMIT if settling else LIMIT):
                ran_out[0] += not settling
                return False
            yield
        return True

    def producer():
        stage, phase, uphase = 0, 1, 1

        def settle(q_too):
            if mistake == "no settling":
                return
            for i in range(stages):
                ok = yield from wait(full[i], phase ^ 1 if i < stage else phase, settling=True)
                assert ok, "the settling itself ran out"
            if q_too or mistake == "Q waited for after the end":
                ok = yield from wait(ufull, uphase, settling=True)
                assert ok, "the settling itself ran out"

        for n, tiles in enumerate(units):
            if not (yield from wait(uempty, uphase)):
                yield from settle(True)
                return
            uphase ^= 1
            unit_now[0] = (n, tiles)
            ufull.arrive(loads=1)
            load(ufull)
            yield
            for t in range(tiles):
                if not (yield from wait(empty[stage], phase)):
                    yield from settle(True)
                    return
                if slots[stage] is not None and not ran_out[0]:
                    assert len(readers[stage]) == warps, "a slot is rewritten before every warp has read it"
                slots[stage], readers[stage] = (n, t), set()
                full[stage].arrive(loads=2)
                load(full[stage])
                load(full[stage])
                yield
                stage += 1
                if stage == stages:
                    stage, phase = 0, phase ^ 1
        freed = yield from wait(uempty, uphase)
        if freed:
            unit_now[0] = (len(units), 0)
            ufull.arrive()
        yield from settle(not freed)

    meeting = [{"in": 0, "round": 0, "dead": False} for _ in range(groups)]

    def consumer(w):
        m = meeting[w // 4]
        stage, phase, uphase, alive = 0, 0, 0, True
        while True:
            if alive:
                alive = yield from wait(ufull, uphase)
            uphase ^= 1
            mine = m["round"]  # the group's barrier
            m["dead"] = m["dead"] or not alive
            m["in"] += 1
            if m["in"] == 4:
                m["in"], m["round"] = 0, mine + 1
            while m["round"] == mine:
                yield
            if m["dead"]:
                return
            n, tiles = unit_now[0]
            if tiles == 0:
                return
            uempty.arrive()
            yield
            for t in range(tiles):
                if alive:
                    alive = yield from wait(full[stage], phase)
                if alive:
                    assert slots[stage] == (n, t)
                    read[w].append((n, t))
                    readers[stage].add(w)
                if alive or mistake == "arriving without having waited":
                    empty[stage].arrive()
                yield
                stage += 1
                if stage == stages:
                    stage, phase = 0, phase ^ 1

    roles = [producer()] + [consumer(w) for w in range(warps)]
    while roles:
        now[0] += 1
        assert now[0] < 100 * LIMIT, "a role does not end"
        for f in [f for f in flying if f[0] <= now[0]]:
            flying.remove(f)
            f[1].land()
        for role in rng.sample(roles, len(roles)):
            if rng.random() < 0.7:
                try:
                    next(role)
                except StopIteration:
                    roles.remove(role)
    assert not flying, "a load is in flight when the CTA ends"
    return ran_out[0], read


CASES = [([3], 3, 1), ([1, 1, 1, 5], 3, 1), ([7, 2, 9], 3, 1), ([2, 1, 6], 6, 2), ([13], 6, 2), ([], 3, 1)]


@pytest.mark.parametrize("units,stages,groups", CASES)
def test_without_slow_loads_nothing_runs_out(units, stages, groups):
    for seed in range(10):
        ran_out, read = run(units, stages, groups, seed)
        assert ran_out == 0
        assert all(r == [(n, t) for n, tiles in enumerate(units) for t in range(tiles)] for r in read)


@pytest.mark.parametrize("units,stages,groups", [c for c in CASES if c[0]])
def test_no_load_outlives_the_cta_when_waits_run_out(units, stages, groups):
    """Every load is the slow one in turn."""
    some = 0
    for slow in range(sum(1 + 2 * t for t in units)):
        for seed in range(3):
            some += run(units, stages, groups, seed, slow)[0]
    assert some > 0


@pytest.mark.parametrize("mistake", ["no settling", "arriving without having waited", "Q waited for after the end"])
def test_planted_mistakes_are_caught(mistake):
    caught = 0
    for units, stages, groups in CASES[:5]:
        for slow in [None] + list(range(sum(1 + 2 * t for t in units))):
            try:
                run(units, stages, groups, 1, slow, mistake)
            except AssertionError:
                caught += 1
    assert caught > 0
