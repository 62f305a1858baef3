"""Attention of drafted tokens where its numbers come to an end: scales, weights that vanish, what is not finite."""
import math
import random

import pytest
import torch

from test_gpu_tree import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("window", [0, 50])
@pytest.mark.parametrize("scale,spread", [(2.0 ** -40, 2.0 ** -112), (2.0 ** -126, 2.0 ** -60), (2.0 ** -20, 2.0 ** -114),
                                          (1e-44, 1.0), (-2.0 ** -40, 2.0 ** -112)])
def test_scores_next_to_nothing(scale, spread, window):
    """Small bf16 queries and scales over an 8-bit cache: all weights are alike, and hidden tokens have none."""
    c = Case([(200, 9), (3, 33), (0, 5), (700, 20)], 4, 2, 64, "bf16", "e4m3", window=window, scale=scale, spread=spread, seed=40)
    c.run().check()


def test_scores_of_zero_under_the_largest_scale():
    """Large bf16 queries whose products with the keys are 0, under a scale next to fp32's largest."""
    c = Case([(200, 9), (3, 33)], 4, 2, 64, "bf16", "e4m3", scale=3.0e38, seed=41)
    c.q.zero_()
    for h in range(4):
        c.q[:, 64 * h] = 2.0 ** 100
    c.k.view(torch.uint8)[..., 0] = 0
    c.run().check()


def far(seqs, tiles, bad, dtype="bf16", kv=None, hq=4, hkv=2, d=64, step=128, **how):
    """Queries and keys such that the tokens of some tiles of 128 have weights below 2^-300, and the value of one
    of those tokens, in column 3, is `bad`.  tiles(b): those of sequence b; the first holds the value."""
    c = Case(seqs, hq, hkv, d, dtype, kv, mask=None, scale=1.0, **how)
    c.q.zero_()
    for h in range(hq):
        c.q[:, d * h] = 16.0
    page = c.page
    for b, (ctx, n) in enumerate(seqs):
        j = torch.arange(ctx + n)
        at = (c.pages[b][j // page].long().cuda(), (j % page).cuda())
        low = torch.zeros(ctx + n, dtype=torch.bool)
        for t in tiles(b):
            low[t * step: (t + 1) * step] = True
        low[ctx:] = False
        first = torch.where(low, -16.0, 0.0)[:, None].expand(-1, hkv)
        keys = c.k.view(torch.uint8 if c.ks is not None else c.k.dtype)
        new = (first / (c.ks.cpu() if c.ks is not None else 1.0)).to(c.k.dtype)
        got = keys[at]
        got[..., 0] = new.view(keys.dtype).cuda()
        keys[at] = got
        chosen = [t for t in tiles(b) if t * step + 5 < ctx]
        c.marked = getattr(c, "marked", []) + [bool(chosen)]
        if chosen:
            tok = chosen[0] * step + 5
            c.v[int(c.pages[b][tok // page]), tok % page, :, 3] = torch.tensor(bad).to(c.v.dtype)
    return c


def look(c, bad):
    """Column 3 is not finite where the value was placed; all else is right."""
    c.run()
    out = c.out.double().view(c.T, c.hq, c.d).clone()
    lse = c.lse.clone()
    for b, (ctx, n) in enumerate(c.seqs):
        rows = slice(c.starts[b], c.starts[b + 1])
        if c.marked[b]:
            col = out[rows, :, 3]
            assert bool((torch.isnan(col) | (col == bad)).all()), (b, ctx, n, col.flatten()[:6])
            c.out.view(c.T, c.hq, c.d)[rows, :, 3] = 0
    assert bool(torch.isfinite(lse).all())
    c.v[..., 3] = 0     # and now the other columns, and the other sequences, by the definition
    keep = c.out.clone()
    for b in range(len(c.seqs)):
        if not c.marked[b]:
            keep.view(c.T, c.hq, c.d)[c.starts[b]: c.starts[b + 1], :, 3] = 0
    c.out = keep
    c.check()


@pytest.mark.parametrize("kv", ["bf16", "fp16", "e4m3"])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_values_of_vanishing_weight_in_a_stream(kv, bad):
    """Short items, whole in a CTA, whose steps two streams share: one has nothing but weights that vanish."""
    if kv == "e4m3" and bad == math.inf:
        pytest.skip("no infinities in E4M3")
    rng = random.Random(7)
    seqs = [(rng.randrange(130, 420), rng.randrange(1, 7)) for _ in range(400)]
    c = far(seqs, lambda b: [b % 2] if seqs[b][0] < 256 else [b % 2, b % 2 + 2], bad, "bf16" if kv == "e4m3" else kv, kv, seed=42)
    look(c, bad)


@pytest.mark.parametrize("kv,hq,d", [("bf16", 4, 64), ("fp16", 16, 128), ("e4m3", 4, 64), ("bf16", 4, 256)])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_values_of_vanishing_weight_in_a_part(kv, hq, d, bad):
    """Long items, cut into parts: whole parts of nothing but weights that vanish."""
    if kv == "e4m3" and bad == math.inf:
        pytest.skip("no infinities in E4M3")
    c = far([(60000, 12)], lambda b: range(20, 300), bad, "bf16" if kv == "e4m3" else kv, kv, hq=hq, d=d, seed=43, page=64)
    look(c, bad)


@pytest.mark.parametrize("kv", ["bf16", "fp16"])
@pytest.mark.parametrize("ctx", [0, 40, 128, 20000])
def test_nan_values_of_infinite_negative_scores(kv, ctx):
    """A weight of 0 times NaN is NaN: in context, and of drafted tokens that have a part of their own."""
    c = Case([(ctx, 5)], 2, 1, 64, kv, mask=lambda n, r: [1 << i for i in range(n)], scale=1.0, seed=44)
    want = c.run().out.clone()
    c.q[:, ::64] = 1.0
    put = [(ctx + 2, [2])] + ([(ctx // 2, range(5))] if ctx else [])
    for tok, rows in put:
        c.k[int(c.pages[0][tok // 16]), tok % 16, 0, 0] = -math.inf
        c.v[int(c.pages[0][tok // 16]), tok % 16, 0, 9 if tok >= ctx else 10] = math.nan
    c.run()
    out = c.out.view(5, 2, 64)
    assert bool(torch.isnan(out[2, :, 9]).all()) and bool(torch.isfinite(out[[0, 1, 3, 4], :, 9]).all())
    if ctx:
        assert bool(torch.isnan(out[..., 10]).all()) and bool(torch.isfinite(c.lse).all())
    others = [x for x in range(64) if x not in (9, 10)]
    assert bool(torch.isfinite(out[..., others][[0, 1, 3, 4]]).all()) and bool(torch.isfinite(want).all())
