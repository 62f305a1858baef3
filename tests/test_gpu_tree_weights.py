"""The tree attention's weights, seen where a row's values cancel: what is left is their error."""
import pytest
import torch

from test_gpu_tree import Case, bits
from test_tree_weights import WEIGHTS

pytestmark = pytest.mark.gpu


def cancelling(kind, seed, tokens=26, count=300):
    """Sequences of one tile whose scores are exact and whose values, by the choice of the last six, add up to next to
    nothing in 64 bits."""
    c = Case([(tokens - 1, 1)] * count, 2, 1, 64, "bf16" if kind == "bf16" else "fp16", kind, mask=None, scale=1.0, seed=seed)
    g = torch.Generator(device="cuda").manual_seed(seed)
    if kind == "e4m3":
        c.ks, c.vs = (torch.ones(1, device="cuda") for _ in range(2))
    c.q.zero_()
    c.q[:, ::64] = 1.0
    # scores: numbers of E4M3, which all types hold; the last six smaller and smaller
    s = (-4 * torch.rand(count, tokens, generator=g, device="cuda")).to(torch.float8_e4m3fn).double()
    s[:, -6:] = torch.arange(-1, -7, -1, device="cuda").double()
    p = s.exp()
    v = (4 * torch.randn(count, tokens, 64, generator=g, device="cuda")).to(c.v.dtype).double()
    rest = (p[:, :-6, None] * v[:, :-6]).sum(1)
    for t in range(tokens - 6, tokens):
        v[:, t] = (-rest / p[:, t, None]).to(c.v.dtype).double()
        rest += p[:, t, None] * v[:, t]
    j = torch.arange(tokens)
    for b in range(count):
        at = (c.pages[b][j // 16].long().cuda(), (j % 16).cuda())
        keys = torch.zeros(tokens, 1, 64, device="cuda")
        keys[:, 0, 0] = s[b]
        bits(c.k)[at] = bits(keys.to(c.k.dtype))
        bits(c.v)[at] = bits(v[b][:, None].to(c.v.dtype))
    total = p.sum(1)[:, None]
    mag = (p[..., None] * v.abs()).sum(1) / total
    return c, rest / total, mag


@pytest.mark.parametrize("kind", WEIGHTS)
def test_weights_are_as_exact_as_stated(kind):
    """Errors of the weights, each of its own sign, add up to at most the bound times sum p |v|.  Besides: four MMAs whose
    fp32 sums may each be cut at 2^-23 of what is added, the factor log2 e (2^-23 of arguments below 9) and the
    output's own rounding.  Most of a lost low part of P would be 2^-9 and more."""
    half = torch.finfo(torch.bfloat16 if kind == "bf16" else torch.float16).eps / 2
    for seed in range(3):
        c, want, mag = cancelling(kind, seed)
        assert bool((want.abs() <= mag * 2.0 ** -20).all())      # they do cancel
        c.run()
        out = c.out.double().view(-1, 2, 64)
        for h in range(2):
            off = (out[:, h] - want).abs()
            bound = mag * (WEIGHTS[kind] + 4 * 2.0 ** -23 + 9 * 2.0 ** -23 * 0.7) + want.abs() * half + 2.0 ** -25
            assert bool((off <= bound).all()), (kind, seed, float((off / mag).max()))
