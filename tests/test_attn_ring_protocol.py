"""The attention kernel's ring of steps, as a model on the CPU.

Producers take the steps of a share in turn (x % PW), consumers those of a segment by their place
in the item, (step + item) % W, and meet at a barrier between segments.  Stage x % NST has a full
and an empty barrier, whose waits only see one bit of the phase.  The model runs producers and
consumers in random order and checks that what a consumer reads is its own step and that no
producer overwrites an unread one."""
import random

import pytest


class Broken(Exception):
    pass


def run(nst, segments, seed, W=8, PW=4):
    """segments: (item, first step, steps) in order.  Raises Broken where the protocol fails."""
    rng = random.Random(seed)
    owner, seg_of = [], []           # consumer and segment of each step
    for k, (item, first, n) in enumerate(segments):
        owner += [(first + j + item) % W for j in range(n)]
        seg_of += [k] * n
    total = len(owner)
    full = [0] * nst                 # completed phases
    empty = [0] * nst
    held = [None] * nst              # step in the stage, and whether it was read
    read = [True] * nst
    prod = list(range(PW))           # next step of each producer
    todo = [[x for x in range(total) if owner[x] == w] for w in range(W)]
    seg = [0] * W                    # the segment each consumer is in
    passed = lambda phases, parity: (phases & 1) != parity  # noqa: E731  (test_wait.parity)
    pace = [rng.choice([1, 1, 1, 8]) for _ in range(W)]
    while any(todo) or any(p < total for p in prod):
        moves = []
        for p in range(PW):
            x = prod[p]
            if x < total and passed(empty[x % nst], ((x // nst) & 1) ^ 1):
                moves.append(("p", p))
        for w in range(W):
            nxt = seg_of[todo[w][0]] if todo[w] else len(segments)
            if seg[w] < nxt:
                # the barrier at a segment's end: everybody has done its steps of it
                if all(not todo[v] or seg_of[todo[v][0]] > seg[w] for v in range(W)):
                    moves.append(("b", w))
            elif todo[w] and passed(full[todo[w][0] % nst], (todo[w][0] // nst) & 1):
                if rng.randrange(pace[w]) == 0:
                    moves.append(("c", w))
        if not moves:
            if any(todo[w] and seg[w] == seg_of[todo[w][0]] and passed(
                    full[todo[w][0] % nst], (todo[w][0] // nst) & 1) for w in range(W)):
                continue             # a slow consumer's turn passed by
            raise Broken("nothing can move")
        kind, who = rng.choice(moves)
        if kind == "p":
            x = prod[who]
            if not read[x % nst]:
                raise Broken(f"step {held[x % nst]} overwritten by {x}")
            held[x % nst], read[x % nst] = x, False
            full[x % nst] += 1
            prod[who] += PW
        elif kind == "b":
            seg[who] += 1
        else:
            x = todo[who].pop(0)
            if held[x % nst] != x or read[x % nst]:
                raise Broken(f"consumer of {x} finds {held[x % nst]}")
            read[x % nst] = True
            empty[x % nst] += 1


def _segments(rng):
    return [(rng.randrange(100), rng.randrange(50), rng.choice([1, 3, 8, 17, 40, 120]))
            for _ in range(rng.randrange(1, 7))]


@pytest.mark.parametrize("nst,W,PW", [(8, 8, 4), (16, 8, 4), (16, 8, 8), (32, 8, 8), (16, 4, 4), (8, 4, 4)])
def test_every_step_is_read_once_by_its_consumer(nst, W, PW):
    for seed in range(150):
        run(nst, _segments(random.Random(seed)), seed, W, PW)


@pytest.mark.parametrize("nst", [22, 23])
def test_other_depths_fail(nst):
    """A depth that is no multiple of PW: a producer passes a wait two rounds early."""
    failed = 0
    for seed in range(150):
        try:
            run(nst, _segments(random.Random(seed)), seed)
        except Broken:
            failed += 1
    assert failed > 0


def test_the_kernel_asserts_what_the_model_needs():
    import os
    src = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                            "weight_only_int4_tma_gb300", "csrc", "attn.cuh")).read()
    assert "static_assert(NST % W == 0 && NST % PW == 0" in src
    assert "W = DP == 256 && NT == 2 ? 4 : 8;" in src
    assert "PW = NT == 1 && DP <= 128 ? 8 : 4;" in src
    assert "NST = (128 << 10) / (2 * SLOT);" in src
