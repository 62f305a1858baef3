"""How the attention kernel cuts the line of items in shares, restated on the CPU: every step of
every item belongs to exactly one CTA, the parts of an item are those of neighbouring CTAs, and
their count and slots are what the kernel computes from the line alone."""
import random

import pytest

COST = 8


def lay(n_steps, items, ctas, join=4, WARPS=8):
    """(end, share, apart, whole items): n_steps of each sequence, items per sequence."""
    seqs = [n for n in n_steps if n]
    total = sum(n + COST for n in seqs) * items
    share, apart = max(-(-total // ctas), 1), False
    count, rounds = len(seqs) * items, -(-share // WARPS)
    if 2 * count <= ctas:
        steps = total - count * COST
        left = (ctas - count) * WARPS
        r = max(-(-steps // left), 1)
        apart = r <= max(-(-steps // (ctas * WARPS)), 1) + 1 + join
        if apart:
            rounds, share = r, r * WARPS
    whole = -(-max(seqs, default=0) // WARPS)
    if count <= ctas and whole < rounds + join + (not apart):
        apart, share = True, max(whole * WARPS, 1)
    over = (join + 2) * WARPS
    return total, share, apart, (count > ctas and max(seqs) + COST <= min(4 * over, share + over) and
                                 -(-count // ctas) * (total // count) <= share + over)


def after(seg, n_steps, items, uncut):
    b, item = seg["b"], seg["item"] + 1
    if item == items:
        item, b = 0, b + 1
        while n_steps[b] == 0 and b + 1 < len(n_steps):
            b += 1
    return dict(b=b, item=item, step=0, end=n_steps[b] if uncut else min(n_steps[b], seg["rest"] - COST), n=n_steps[b],
                rest=seg["rest"] - COST - n_steps[b])


def locate(cta, n_steps, items, end, share, apart, uncut):
    if apart:
        done = 0
        for b, n in enumerate(n_steps):
            per = -(-n // share)
            if done <= cta < done + per * items:
                step = (cta - done) % per * share
                return dict(b=b, item=(cta - done) // per, step=step, end=min(n, step + share), n=n, rest=0)
            done += per * items
        return None
    u, stop = share * cta, min(end, share * (cta + 1))
    if u >= end:
        return None
    at, b = 0, 0
    length = lambda b: (n_steps[b] + COST) * items if n_steps[b] else 0  # noqa: E731
    while at + length(b) <= u and b + 1 < len(n_steps):
        at += length(b)
        b += 1
    n = n_steps[b]
    item = (u - at) // (n + COST)
    begin = at + item * (n + COST)
    rest = stop - begin - COST - n
    seg = dict(b=b, item=item, step=max(u - begin - COST, 0), end=min(n, n + rest), n=n, rest=rest)
    if uncut:
        seg["end"] = n
    if u == begin if uncut else seg["step"] < seg["end"]:
        return seg
    return after(seg, n_steps, items, uncut) if rest > (0 if uncut else COST) else None


def segments(cta, n_steps, items, line):
    """[(segment, first CTA and number of the item's parts)]"""
    end, share, apart, uncut = line
    seg, got = locate(cta, n_steps, items, *line), []
    if seg is None:
        return got
    begin = min(end, share * (cta + 1)) - seg["rest"] - COST - seg["n"]
    while True:
        assert 0 <= seg["step"] < seg["end"] <= seg["n"]
        if seg["step"] == 0 and seg["end"] == seg["n"]:
            c0, n = cta, 1
        elif apart:
            c0, n = cta - seg["step"] // share, -(-seg["n"] // share)
        else:
            c0 = (begin + COST) // share
            n = (begin + COST + seg["n"] - 1) // share - c0 + 1
        got.append((seg, c0, n))
        if seg["rest"] <= (0 if uncut else COST):
            return got
        begin += COST + seg["n"]
        seg = after(seg, n_steps, items, uncut)


@pytest.mark.parametrize("seed", range(400))
def test_every_step_belongs_to_one_cta(seed):
    rng = random.Random(seed)
    ctas = rng.choice([1, 2, 7, 152])
    longest = rng.choice([1, 8, 30, 64, 3000])
    n_steps = [min(longest, rng.choice([0, 1, 2, 5, 40, rng.randrange(1, 3000)])) for _ in range(rng.randrange(1, 60))]
    items = rng.choice([1, 2, 8, 32])
    line = lay(n_steps, items, ctas, rng.choice([0, 3, 4]), rng.choice([4, 8]))
    parts = {}
    for cta in range(ctas):
        segs = segments(cta, n_steps, items, line)
        cut = [(s["step"] == 0, s) for s, _, n in segs if not (s["step"] == 0 and s["end"] == s["n"])]
        assert len({begins for begins, _ in cut}) == len(cut) <= 2   # a slot each
        for s, c0, n in segs:
            parts.setdefault((s["b"], s["item"]), []).append((cta, s["step"], s["end"], c0, n))
    want = {(b, i) for b, n in enumerate(n_steps) if n for i in range(items)}
    assert set(parts) == want
    for (b, i), p in parts.items():
        assert [x[1] for x in p] == [0] + [x[2] for x in p[:-1]] and p[-1][2] == n_steps[b]
        assert all((c0, n) == (p[0][0], len(p)) for _, _, _, c0, n in p)
        assert [x[0] for x in p] == list(range(p[0][0], p[0][0] + len(p)))


def test_one_long_item_among_short_ones_is_cut():
    line = lay([700] + [9] * 40, 8, 152)
    assert not line[2] and not line[3]
    assert max(sum(s["end"] - s["step"] for s, _, _ in segments(c, [700] + [9] * 40, 8, line))
               for c in range(152)) <= line[1]


def test_shares_are_even():
    """Steps and items of the fullest CTA against the mean, for lengths that differ greatly."""
    rng = random.Random(1)
    n_steps = [rng.choice([1, 3, 700]) for _ in range(300)]
    line = lay(n_steps, 8, 152)
    loads = [sum(s["end"] - s["step"] + COST for s, _, _ in segments(c, n_steps, 8, line)) for c in range(152)]
    assert max(loads) <= 1.1 * sum(loads) / 152
