"""The split of the tree attention's work (csrc/tree.cuh), restated: every step of every item is one CTA's, and
the parts of a cut item stand where the join looks for them."""
import random

import pytest

STEP, DUAL, ITEM = 2, 3, 6     # units of a step, of a step of two tiles, of an item by itself


def segments(items, ctas):
    """items: (steps, weight).  Per CTA: (item, first step, end), and for the CTA that begins a cut item the
    number of CTAs that it says hold it."""
    total = sum(s * w + ITEM for s, w in items)
    share = max(-(-total // ctas), DUAL if any(w == DUAL for _, w in items) else STEP)
    out, joins = [], {}
    for cta in range(ctas):
        u, end, mine, at = share * cta, min(total, share * (cta + 1)), [], 0
        for n, (steps, w) in enumerate(items):
            first = at + ITEM
            if u < total and at + steps * w + ITEM > u and at < end:
                before = lambda to: -(-min(max(to - first, 0), steps * w) // w)  # noqa: E731
                lo, hi = before(u), before(end)
                if lo < hi:
                    mine.append((n, lo, hi))
                    if lo == 0 and hi < steps:
                        joins[n] = (cta, (first + (steps - 1) * w) // share - cta + 1)
            at += steps * w + ITEM
        out.append(mine)
    return out, joins


@pytest.mark.parametrize("kind", ["short", "mixed", "one", "long"])
def test_split(kind):
    for seed in range(150):
        rng = random.Random(seed)
        ctas = rng.choice([1, 2, 7, 152])
        count = {"short": 300, "mixed": 60, "one": 1, "long": 5}[kind]
        most = {"short": 3, "mixed": 40, "one": 300, "long": 3000}[kind]
        items = [(rng.randrange(1, most + 1), rng.choice([STEP, DUAL]) if seed % 3 else STEP)
                 for _ in range(rng.randrange(1, count + 1))]
        out, joins = segments(items, ctas)
        held = {}
        for cta, mine in enumerate(out):
            for place, (n, lo, hi) in enumerate(mine):
                held.setdefault(n, []).append((cta, lo, hi))
                if lo > 0:
                    assert place == 0, "a part that another CTA began is a CTA's first"
                if hi < items[n][0]:
                    assert place == len(mine) - 1, "one that is left to a later CTA is its last"
        for n, (steps, _) in enumerate(items):
            parts = held[n]
            assert [p[1] for p in parts] == [0] + [p[2] for p in parts[:-1]] and parts[-1][2] == steps
            assert [p[0] for p in parts] == list(range(parts[0][0], parts[0][0] + len(parts))), "no CTA between has none"
            if len(parts) > 1:
                assert joins[n] == (parts[0][0], len(parts))
            else:
                assert n not in joins
