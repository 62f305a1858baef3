"""The hand-overs of the tree attention's loaders where no tensor map describes the pages (csrc/tree.cuh, 16-bit
caches), restated and run on the CPU with the other roles of test_tree_protocol.

Every loader warp copies its own tokens of each tile into the ring, in groups of asynchronous copies, and arrives for a
tile when its group has landed, two tiles later or as soon as it would have to wait for a slot; tiles with
values that some row does not see are written at once.
"""
import random

import pytest

from test_tree_protocol import Bar, Kernel


class Pieces(Kernel):
    """queries: "copied" (a tensor copy, for which the second loader alone waits) or "pieces" (by all loaders), the same
    for all items, as the scale's sign and the heads decide it: a loader that had not waited in the items before
    could not tell the phases of q_empty apart."""
    LOADERS = 2

    def __init__(self, segs, streams, nslot, queries, rng):
        super().__init__(segs, streams, nslot, rng)
        self.full = [Bar(self.LOADERS) for _ in range(nslot)]
        self.queries, self.shares = queries, [{} for _ in range(nslot)]

    def loading(self):
        return [self.pieces(lw) for lw in range(self.LOADERS)]

    def begin(self, slot, lw):
        """A warp starts to write its share of a tile."""
        self.slots[slot] = "loading"
        assert lw not in self.shares[slot], "its share of the tile before is complete and read"

    def landed(self, slot, lw, what):
        self.shares[slot][lw] = what
        if len(self.shares[slot]) == self.LOADERS:
            assert len(set(self.shares[slot].values())) == 1, self.shares[slot]
            self.slots[slot], self.shares[slot] = what, {}

    def settle(self, under_way):
        """Waits for all groups, oldest first, and arrives for each."""
        for group, slot in under_way:
            yield group, 0
            self.full[slot].arrive()
        under_way.clear()

    def before_waiting(self, under_way):
        yield from self.settle(under_way)

    def pieces(self, lw):
        slot, phase, q_phase, g = 0, 0, 0, 0
        for n, (steps, _, unclean) in enumerate(self.segs):
            under_way = []          # (its landing, slot) of the groups that nobody has arrived for
            for st in range(steps):
                for side in range(2):
                    what = ("KV"[side], g, True)
                    if not self.empty[slot].passes(phase ^ 1):
                        yield from self.before_waiting(under_way)
                        yield self.empty[slot], phase ^ 1
                    self.begin(slot, lw)
                    if side and st in unclean:
                        yield None
                        self.landed(slot, lw, what)
                        self.full[slot].arrive()
                    else:
                        group = Bar(1)

                        def land(slot=slot, what=what, group=group):
                            self.landed(slot, lw, what)
                            group.arrive()
                        self.after(land)
                        under_way.append((group, slot))
                        if len(under_way) > 2:      # the oldest of three: all but two have landed
                            first = under_way.pop(0)
                            yield first[0], 0
                            self.full[first[1]].arrive()
                    slot, phase = (slot + 1) % self.nslot, phase ^ (slot + 1 == self.nslot)
                if st == 0:
                    yield from self.settle(under_way)
                    if self.queries == "copied":
                        if lw == 1:
                            yield self.q_empty, q_phase ^ 1
                            self.q = "loading"

                            def put_q(n=n):
                                self.q = n
                                self.q_full.complete(1)
                            self.q_full.arrive(1)
                            self.after(put_q)
                    else:
                        yield self.q_empty, q_phase ^ 1
                        self.q = "loading"
                        yield None
                        yield self.loaders
                        if lw == 0:
                            self.q = n
                            self.q_full.arrive()
                    q_phase ^= 1
                g += 1
            yield from self.settle(under_way)


def batch(rng, streams):
    segs = []
    for _ in range(rng.randrange(1, 9)):
        steps = rng.choice([1, 1, 1, 2, 3, rng.randrange(1, 12)])
        unclean = {st for st in range(steps) if rng.random() < (0.8 if st == steps - 1 else 0.1)}
        segs.append((steps, streams == 2 and rng.random() < 0.5, unclean))
    return segs


@pytest.mark.parametrize("streams,nslot", [(2, 4), (2, 8), (1, 4)])
def test_hand_overs_in_pieces(streams, nslot):
    for seed in range(120):
        rng = random.Random(seed)
        segs = batch(rng, streams)
        Pieces(segs, streams, nslot, rng.choice(["copied", "pieces"]), rng).run()


def found(kind, seeds=40):
    count = 0
    for seed in range(seeds):
        rng = random.Random(seed)
        segs = batch(rng, 2)
        try:
            kind(segs, 2, 4, "copied", rng).run()
        except AssertionError:
            count += 1
    return count


def test_the_model_sees_tiles_that_are_never_announced():
    """A warp that waits for a slot before it has arrived for what it holds back may wait for itself."""
    class Holding(Pieces):
        def before_waiting(self, under_way):
            yield None

    class Forgetting(Pieces):
        def settle(self, under_way):
            yield None
            under_way.clear()
    assert found(Pieces) == 0 and found(Forgetting) > 30
    assert found(Holding, 300) > 2      # (two tiles held back of a ring of four: rarely what all wait for)


def test_the_model_sees_an_early_announcement():
    """Arriving for a tile before its copies have landed."""

    class Early(Pieces):
        def settle(self, under_way):
            yield None
            for _, slot in under_way:
                self.full[slot].arrive()
            under_way.clear()
    assert found(Early) > 10
