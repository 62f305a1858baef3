"""The 64-bit statements of oracle/drafts.py, pinned by hand-made numbers and by torch."""
import math

import torch

from oracle import drafts


def test_seen():
    # a root, two children, a grandchild of the first: 1, 3, 5, 11
    assert drafts.seen(2, 4, [1, 3, 5, 11], 0, 0) == [[0, 1, 2], [0, 1, 2, 3], [0, 1, 2, 4], [0, 1, 2, 3, 5]]
    # a window of three tokens on each path, one sink
    assert drafts.seen(5, 4, [1, 3, 5, 11], 3, 1) == [[0, 3, 4, 5], [0, 4, 5, 6], [0, 4, 5, 7], [0, 5, 6, 8]]
    assert drafts.seen(3, 3, None, 2, 0) == [[2, 3], [3, 4], [3, 4, 5]]
    assert drafts.seen(0, 2, [0, 2], 0, 4) == [[], [1]]


def test_attn_row():
    g = torch.Generator().manual_seed(0)
    q, k, v = (torch.randn(n, 8, generator=g, dtype=torch.float64) for n in (3, 20, 20))
    out, lse, mag, spread = drafts.attn_row(q, k, v, 0.3)
    p = torch.softmax(0.3 * q @ k.T, 1)
    assert torch.allclose(out, p @ v) and torch.allclose(mag, p @ v.abs())
    assert torch.allclose(lse, torch.logsumexp(0.3 * q @ k.T, 1))
    out, lse, _, _ = drafts.attn_row(q, k[:0], v[:0], 0.3)
    assert bool((out == 0).all()) and bool((lse == -math.inf).all())


def test_order():
    x = torch.tensor([0.0, 2.0, -0.0, math.nan, 2.0, -math.inf, math.inf])
    assert drafts.order(x) == [3, 6, 1, 4, 0, 2, 5]


def test_logprob_row():
    x = torch.randn(50, generator=torch.Generator().manual_seed(1))
    logp, lse, ent = drafts.logprob_row(x, 0.7)
    want = torch.log_softmax(x.double() * 0.7, 0)
    assert torch.allclose(logp, want) and math.isclose(ent, float(-(want.exp() * want).sum()))
    assert math.isclose(lse, float(torch.logsumexp(x.double() * 0.7, 0)))
    x[3] = -math.inf
    logp, lse, ent = drafts.logprob_row(x, 1.0)
    assert logp[3] == -math.inf and math.isfinite(ent)
    assert drafts.logprob_row(torch.full((4,), -math.inf), 1.0)[1:] == (-math.inf, 0.0)
    logp, lse, ent = drafts.logprob_row(torch.tensor([1.0, math.inf]), 1.0)
    assert logp[0] == -math.inf and math.isnan(logp[1]) and lse == math.inf and math.isnan(ent)
    assert math.isnan(drafts.logprob_row(x, 0.0)[1]) and math.isnan(drafts.logprob_row(x, math.inf)[1])


def test_move():
    c = torch.arange(12).view(3, 4, 1, 1)
    got = drafts.move(c, [5, 1, 0, -1, 99], [1, 2, 1, 3, 4], [0, 3, 5], 4)
    assert got.flatten().tolist() == [0, 0, 5, 3, 4, 5, 6, 7, 8, 9, 10, 11]
