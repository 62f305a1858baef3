"""The hand-overs of the tree attention's roles (csrc/tree.cuh), restated and run on the CPU.

Loaders, the MMAs' warps and the softmax warps meet at mbarriers, whose waits see one bit of phase.
The model runs the roles in random order, completes copies and MMAs after random times, and checks that
whoever reads a slot of the ring, a place of S and P, or O finds what it is meant to, that nothing is
overwritten before it was read, and that all end.
"""
import random

import pytest


class Bar:
    """An mbarrier: a wait for parity p passes once the phase with that parity is complete."""

    def __init__(self, count):
        self.count, self.pending, self.tx, self.phase = count, count, 0, 0

    def arrive(self, tx=0):
        assert self.pending > 0, "more arrivals than the phase expects"
        self.pending -= 1
        self.tx += tx
        self.settle()

    def complete(self, tx):
        self.tx -= tx
        self.settle()

    def settle(self):
        if self.pending == 0 and self.tx == 0:
            self.phase ^= 1
            self.pending = self.count

    def passes(self, parity):
        return self.phase != parity


class Sync:
    """A named barrier of n agents."""

    def __init__(self, n):
        self.n, self.waiting, self.round = n, 0, 0

    def enter(self):
        self.waiting += 1
        mine = self.round
        if self.waiting == self.n:
            self.waiting, self.round = 0, self.round + 1
        return mine


class Kernel:
    def __init__(self, segs, streams, nslot, rng):
        self.segs, self.streams, self.nslot, self.rng = segs, streams, nslot, rng
        self.full = [Bar(1) for _ in range(nslot)]
        self.empty = [Bar(streams) for _ in range(nslot)]
        sw = 4 * streams
        self.q_full, self.q_empty = Bar(1), Bar(streams + sw)
        self.s_full, self.p_full = [Bar(2) for _ in range(2)], [Bar(4) for _ in range(2)]
        self.turn = [Bar(1), Bar(1)]
        self.o_full, self.o_free, self.pv_done, self.fix = Bar(2 * streams), Bar(sw), Bar(1), Bar(1)
        self.loaders, self.softmaxes = Sync(2), Sync(sw)
        self.slots, self.q = [None] * nslot, None
        self.places = [None, None]                 # ("S", step, stream) or {"P": ..., halves}
        self.o = [[] for _ in range(streams)]
        self.later = []                            # (time, action) in flight
        self.queues = [[] for _ in range(streams)]  # an MMA thread's operations, in order
        self.time, self.results = 0, []

    def after(self, action):
        self.later.append((self.time + self.rng.randrange(1, 60), action))

    def loading(self):
        return [self.loader(0), self.loader(1)]

    # ---- the loaders: keys by the first, queries and values by the second ----
    def loader(self, lw):
        slot, phase, q_phase, fix_phase, g = 0, 0, 0, 0, 0
        for n, (steps, dual, unclean) in enumerate(self.segs):
            if lw == 1:
                yield self.q_empty, q_phase ^ 1

                def put_q(n=n):
                    self.q = n
                    self.q_full.complete(1)
                self.q = "loading"
                self.q_full.arrive(1)
                self.after(put_q)
            q_phase ^= 1
            for st in range(steps):
                mine, clean = slot + lw, st not in unclean
                yield self.empty[mine], phase ^ 1
                bar = self.full[mine] if clean or lw == 0 else self.fix

                def put(mine=mine, what=("KV"[lw], g, clean or lw == 0), bar=bar):
                    self.slots[mine] = what
                    bar.complete(1)
                self.slots[mine] = "loading"
                bar.arrive(1)
                self.after(put)
                if not clean:
                    if lw == 1:
                        yield self.fix, fix_phase
                        fix_phase ^= 1
                    yield self.loaders
                    yield self.loaders
                    if lw == 1:
                        assert self.slots[mine] == ("V", g, False)
                        self.slots[mine] = ("V", g, True)
                        self.full[mine].arrive()
                slot, phase, g = (slot + 2) % self.nslot, phase ^ (slot + 2 >= self.nslot), g + 1

    # ---- the MMAs of a stream ----
    def mma(self, stream):
        q_phase, free_phase, p_phase, step0, turns = 0, 0, [0, 0], 0, 0
        queue = self.queues[stream]
        for n, (steps, dual, _) in enumerate(self.segs):
            alone = self.streams == 2 and not dual
            first, stride = ((stream ^ step0) & 1, 2) if alone else (0, 1)
            yield self.q_full, q_phase
            q_phase ^= 1

            def keys(st):
                at = step0 + st
                return self.full[2 * at % self.nslot], (2 * at // self.nslot) & 1

            def scores(st):
                at = step0 + st
                slot, place = 2 * at % self.nslot, stream if self.streams == 2 else at & 1
                yield keys(st)

                def run(at=at, slot=slot, place=place, n=n):
                    assert self.slots[slot] == ("K", at, True), (self.slots[slot], at)
                    assert self.q == n, "the queries of this item"
                    assert self.places[place] is None, "P V of what stood here is done"
                    self.places[place] = ("S", at, stream)
                queue.append(run)
                queue.append(self.s_full[place].arrive)
                queue.append(self.empty[slot].arrive)
                if alone:
                    queue.append(self.empty[slot].arrive)
                if st + stride >= steps:
                    queue.append(self.q_empty.arrive)
                self.s_full[place].arrive()

            if first >= steps:
                self.q_empty.arrive()
                yield self.o_free, free_phase ^ 1
                free_phase ^= 1
                self.o_full.arrive()
                self.o_full.arrive()
            for st in range(first - stride, steps, stride):
                again = st + stride < steps
                if self.streams == 1 and again:
                    yield from scores(st + stride)
                if st >= first:
                    at = step0 + st
                    slot, place = 2 * at % self.nslot + 1, stream if self.streams == 2 else at & 1
                    if st == first:
                        yield self.o_free, free_phase ^ 1
                        free_phase ^= 1
                    yield self.full[slot], (2 * at // self.nslot) & 1
                    yield self.p_full[place], p_phase[place]
                    p_phase[place] ^= 1
                    if dual:
                        yield self.turn[stream], (turns & 1) ^ (stream == 0)

                    def run(at=at, slot=slot, place=place, fresh=st == first):
                        assert self.slots[slot] == ("V", at, True), (self.slots[slot], at)
                        p = self.places[place]
                        assert isinstance(p, dict) and p["at"] == at and p["done"] == 4, (p, at)
                        if fresh:
                            self.o[stream] = []
                        self.o[stream].append(at)
                        self.places[place] = None
                    queue.append(run)
                    queue.append(self.empty[slot].arrive)
                    if alone:
                        queue.append(self.empty[slot].arrive)
                    if self.streams == 1:
                        queue.append(self.pv_done.arrive)
                    if st + stride >= steps:
                        queue.append(self.o_full.arrive)
                        self.o_full.arrive()
                    if dual:
                        there = again and keys(st + 1)[0].passes(keys(st + 1)[1])
                        if there:
                            yield from scores(st + 1)
                        self.turn[stream ^ 1].arrive()
                        turns += 1
                        if again and not there:
                            yield from scores(st + 1)
                        continue
                if self.streams == 2 and again:
                    yield from scores(st + stride)
            step0 += steps

    # ---- a softmax warp ----
    def softmax(self, stream):
        s_phase, o_phase, step0, jobs = [0, 0], 0, 0, 0
        for n, (steps, dual, _) in enumerate(self.segs):
            alone = self.streams == 2 and not dual
            first = (stream ^ step0) & 1 if alone else 0
            if first >= steps:
                self.q_empty.arrive()
            for st in range(first, steps, 2 if alone else 1):
                at = step0 + st
                place = stream if self.streams == 2 else at & 1
                yield self.s_full[place], s_phase[place]
                s_phase[place] ^= 1
                if st == first:
                    assert self.q == n, "the queries' exponents"
                    self.q_empty.arrive()
                elif self.rng.random() < 0.3:  # a new reference: O is scaled, which nothing else touches now
                    if self.streams == 1:
                        yield self.pv_done, (jobs - 1) & 1
                    before = at - (2 if alone else 1)
                    assert self.o[stream][-1] == before, (self.o[stream], before)
                p = self.places[place]
                if isinstance(p, tuple):
                    assert p == ("S", at, stream), (p, at)
                    p = self.places[place] = {"at": at, "done": 0}
                assert p["at"] == at
                p["done"] += 1
                yield None
                self.p_full[place].arrive()
                jobs += 1
            yield self.o_full, o_phase
            o_phase ^= 1
            if alone:
                yield self.softmaxes
            for x in range(self.streams):
                mine = range(step0, step0 + steps) if not alone else \
                    [at for at in range(step0, step0 + steps) if at & 1 == x]
                if (alone or x == stream) and len(mine):
                    assert self.o[x] == list(mine), (x, self.o[x], mine)
            yield None
            self.o_free.arrive()
            step0 += steps
        self.results.append(step0)

    def run(self):
        agents = self.loading() + [self.mma(s) for s in range(self.streams)]
        agents += [self.softmax(s) for s in range(self.streams) for _ in range(4)]
        state = [(a, None) for a in agents]       # what each waits for
        favour = [self.rng.random() ** 3 for _ in agents]
        idle = 0
        while any(a is not None for a, _ in state) or self.later or any(self.queues):
            self.time += 1
            moved = False
            for entry in [e for e in self.later if e[0] <= self.time]:
                self.later.remove(entry)
                entry[1]()
                moved = True
            for q in self.queues:
                if q and self.rng.random() < 0.4:
                    q.pop(0)()
                    moved = True
            for i, (a, need) in enumerate(state):
                if a is None or self.rng.random() > 0.05 + favour[i]:
                    continue
                if isinstance(need, tuple) and isinstance(need[0], Bar) and not need[0].passes(need[1]):
                    continue
                if isinstance(need, tuple) and isinstance(need[0], Sync) and need[0].round == need[1]:
                    continue
                try:
                    need = next(a)
                    if isinstance(need, Sync):
                        need = (need, need.enter())
                    state[i] = (a, need)
                except StopIteration:
                    state[i] = (None, None)
                moved = True
            idle = 0 if moved else idle + 1
            assert idle < 2000, "nobody moves"
        assert len(self.results) == 4 * self.streams


class Converting(Kernel):
    """With an 8-bit cache: a warp copies raw tiles, the others convert them into the ring.  queries: for each
    item how they come: "raw" (copied, then converted by all), "copied", or "pieces" (by all).  late: a
    tile is announced when the next one's copies are under way (pages without tensor maps)."""
    CONVERTERS = 3

    def __init__(self, segs, streams, nslot, nraw, queries, late, rng):
        super().__init__(segs, streams, nslot, rng)
        self.nraw, self.queries, self.late = nraw, queries, late
        self.raw, self.q_raw, self.converters = [None] * nraw, Bar(1), Sync(self.CONVERTERS)
        self.raw_full, self.raw_empty, self.landed = ([Bar(1) for _ in range(nraw)] for _ in range(3))

    def loading(self):
        return [self.copier()] + [self.converter(c) for c in range(self.CONVERTERS)]

    def copier(self):
        at, phase, g = 0, 0, 0
        for steps, _, _ in self.segs:
            before = None
            for half in range(2 * steps):
                yield self.raw_empty[at], phase ^ 1
                assert self.raw[at] in (None, "read")
                self.raw[at] = "loading"

                def put(at=at, what=("KV"[half & 1], g + half // 2)):
                    self.raw[at] = what
                    if self.late:
                        self.landed[at].arrive()
                    else:
                        self.raw_full[at].complete(1)
                if not self.late:
                    self.raw_full[at].arrive(1)
                self.after(put)
                if self.late and before:
                    yield self.landed[before[0]], before[1]
                    self.raw_full[before[0]].arrive()
                before = (at, phase)
                at, phase = (at + 1) % self.nraw, phase ^ (at + 1 == self.nraw)
            if self.late:
                yield self.landed[before[0]], before[1]
                self.raw_full[before[0]].arrive()
            g += steps

    def converter(self, c):
        slot, phase, at, raw_phase, q_phase, g = 0, 0, 0, 0, 0, 0
        for n, (steps, _, _) in enumerate(self.segs):
            how = self.queries[n]
            if how != "pieces" and c == 0:
                yield self.q_empty, q_phase ^ 1
                bar = self.q_raw if how == "raw" else self.q_full

                def put_q(what=("raw", n) if how == "raw" else n, bar=bar):
                    self.q = what
                    bar.complete(1)
                self.q = "loading"
                bar.arrive(1)
                self.after(put_q)
            for half in range(2 * steps):
                yield self.empty[slot], phase ^ 1
                yield self.raw_full[at], raw_phase
                assert self.raw[at] == ("KV"[half & 1], g + half // 2)
                self.slots[slot] = "loading"
                yield self.converters
                if c == 0:
                    self.slots[slot], self.raw[at] = (*self.raw[at], True), "read"
                    self.full[slot].arrive()
                    self.raw_empty[at].arrive()
                slot, phase = (slot + 1) % self.nslot, phase ^ (slot + 1 == self.nslot)
                at, raw_phase = (at + 1) % self.nraw, raw_phase ^ (at + 1 == self.nraw)
                if half == 0:   # behind the first keys
                    if how == "raw":
                        yield self.q_raw, q_phase
                        assert self.q == ("raw", n)
                    if how == "pieces":
                        yield self.q_empty, q_phase ^ 1
                        self.q = "loading"
                    q_phase ^= 1
                    if how != "copied":
                        yield self.converters
                        if c == 0:
                            self.q = n
                            self.q_full.arrive()
            g += steps


@pytest.mark.parametrize("late", [False, True])
@pytest.mark.parametrize("streams,nslot,nraw", [(2, 4, 2), (2, 8, 4), (1, 4, 2)])
def test_hand_overs_with_conversion(streams, nslot, nraw, late):
    for seed in range(90):
        rng = random.Random(seed)
        segs = []
        for _ in range(rng.randrange(1, 9)):
            steps = rng.choice([1, 1, 1, 2, 3, rng.randrange(1, 12)])
            segs.append((steps, streams == 2 and rng.random() < 0.5, set()))
        ways = rng.choice([["raw"], ["pieces"], ["copied", "pieces"]])
        Converting(segs, streams, nslot, nraw, [rng.choice(ways) for _ in segs], late, rng).run()


@pytest.mark.parametrize("streams,nslot", [(2, 4), (2, 8), (1, 4)])
def test_hand_overs(streams, nslot):
    for seed in range(120):
        rng = random.Random(seed)
        segs = []
        for _ in range(rng.randrange(1, 9)):
            steps = rng.choice([1, 1, 1, 2, 3, rng.randrange(1, 12)])
            unclean = {st for st in range(steps) if rng.random() < (0.8 if st == steps - 1 else 0.1)}
            segs.append((steps, streams == 2 and rng.random() < 0.5, unclean))
        Kernel(segs, streams, nslot, rng).run()


def test_the_model_sees_an_early_arrival():
    """The mistake that the order of o_free and o_full avoids is one that the model finds."""
    class Early(Kernel):
        def mma(self, stream):
            inner = super().mma(stream)
            for need in inner:
                if isinstance(need, tuple) and need[0] is self.o_free:
                    continue               # does not wait for the previous item's readers
                yield need
    found = 0
    for seed in range(60):
        rng = random.Random(seed)
        segs = [(rng.choice([1, 1, 2, 3]), False, set()) for _ in range(8)]
        try:
            Early(segs, 2, 4, rng).run()
        except AssertionError:
            found += 1
    assert found > 10

