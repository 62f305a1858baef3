"""Log probabilities at the ends of the types' ranges: logits further apart than fp32 reaches, small factors."""
import math

import pytest
import torch

import weight_only_int4_tma_gb300 as w4
from oracle import drafts

from test_gpu_logprob import KINDS, call

pytestmark = pytest.mark.gpu

MOST = torch.finfo(torch.float32).max


def close(got, want, size):
    """fp32 results: half a step of the result, the errors of logits times the factor (2^-24 of `size`, twice) and
    of exponentials and sums (2^-20); what fp32 does not reach is infinite."""
    got = got.double().cpu()
    want = torch.as_tensor(want, dtype=torch.float64)
    out = want.abs() >= MOST * (1 + 2.0 ** -25)
    want = torch.where(out, want.sign() * math.inf, want)
    same = (got == want) | (torch.isnan(got) & torch.isnan(want))
    # next to the border either side of it is half a step away
    edge = (want.abs() >= MOST * (1 - 2.0 ** -22)) & (got.abs() >= MOST * (1 - 2.0 ** -22)) & (got.sign() == want.sign())
    off = torch.where(same | edge, torch.zeros_like(got), (got - want).abs())
    bound = torch.where(out, torch.zeros_like(want), want.abs()) * 2.0 ** -23 + size * 2.0 ** -22 + 2.0 ** -20
    assert bool((off <= bound).all()), (got[~(off <= bound)][:5], want[~(off <= bound)][:5])


def statement(row, f):
    """(log probabilities, lse, entropy) in 64 bits, from differences to the largest logit: beside numbers z of 1e38
    even 64 bits do not hold the ln 7 of seven equal largest ones."""
    x = row.double()
    d = (x - x.max()) * f
    total = torch.exp(d).sum()
    p = torch.exp(d) / total
    return d - total.log(), float(x.max() * f + total.log()), float(total.log() - (p * d).sum())


def check(x, factor, ids, top, got):
    lp, lse, ent, tid, tlp = got
    for t in range(x.shape[0]):
        row, f = x[t].cpu(), float(factor[t])
        logp, want_lse, want_ent = statement(row, f)
        size = min(float(row.double().abs().max()) * f, MOST)
        close(lse[t], want_lse, size)
        close(ent[t], want_ent, 30.0)  # its terms are p |z - lse|, which no large z enters
        close(lp[t], logp[ids[t].long().cpu()], size)
        order = drafts.order(row)[:top]
        assert tid[t].tolist() == order, t
        close(tlp[t], logp[order], size)


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
@pytest.mark.parametrize("V", [2, 5, 3001, 70000])
def test_logits_further_apart_than_fp32_reaches(kind, V):
    """Differences of logits pass fp32's largest number; times the factor they are small again."""
    g = torch.Generator(device="cuda").manual_seed(V)
    f = torch.tensor([1e-38, 2.0 ** -126, 3e-38, 1e-37, 2e-40, 0.3, 0.5, 0.7, 1.0, 1.7], device="cuda")
    x = (torch.rand(10, V, generator=g, device="cuda") * 2 - 1) * 3.3e38
    x[:, 0], x[:, 1] = 3e38, -3e38
    x[3, 0], x[3, -1] = -3e38, 3.35e38
    x = x.to(KINDS[kind][0])
    ids = torch.tensor([[0, 1, V - 1]] * 10, dtype=torch.int32, device="cuda")
    check(x, f, ids, 2, call(x, kind, f, ids, 2))


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
@pytest.mark.parametrize("order", ["ascending", "descending"])
def test_references_that_move_far(kind, order):
    """The largest logit comes first or last, over the whole range of the type, in one thread's pieces and over all."""
    for V in (50, 40000, 270000):
        x = torch.linspace(-3.38e38, 3.38e38, V, dtype=torch.float64, device="cuda").to(KINDS[kind][0])[None]
        x = (x if order == "ascending" else x.flip(1)).contiguous()
        ids = torch.tensor([[0, V // 2, V - 1]], dtype=torch.int32, device="cuda")
        for f in (1e-38, 3e-37, 2.0 ** -125):
            factor = torch.tensor([f], device="cuda")
            check(x, factor, ids, 1, call(x, kind, factor, ids, 1))


def test_two_logits_at_both_ends():
    """z = 3 and -3."""
    x = torch.tensor([[3e38, -3e38]], device="cuda")
    f = torch.tensor([1e-38], device="cuda")
    lp, lse, ent, _, _ = call(x, "fp32", f, torch.tensor([[0, 1]], dtype=torch.int32, device="cuda"))
    assert abs(float(lse) - 3.00247569) < 1e-5 and abs(float(ent) - 0.0173135) < 1e-5
    assert abs(float(lp[0, 0]) + 0.00247569) < 1e-5 and abs(float(lp[0, 1]) + 6.00247569) < 1e-5


def test_entropy_is_not_negative():
    """Rows of one certain token, at every place of a thread's order and over smaller ones that come first."""
    g = torch.Generator(device="cuda").manual_seed(1)
    for V in (1, 3, 900, 20000):
        x = torch.randn(400, V, generator=g, device="cuda")
        at = torch.randint(0, V, (400, 1), generator=g, device="cuda")
        x.scatter_(1, at, torch.linspace(3, 120, 400, device="cuda")[:, None])
        lse, ent = call(x, "fp32")[1:3]
        assert bool((ent >= 0).all()) and bool((ent[-50:] < 1e-6).all())
