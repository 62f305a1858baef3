"""The operators of drafted tokens of include/decode.h in 64 bits -- TEST INFRASTRUCTURE ONLY.

Plain statements (torch, float64, a row at a time) of the attention of drafted tokens, of the log
probabilities and of the cache moves.  They run on any device and share no code with the CUDA
library.
"""
from __future__ import annotations

import math

import torch

F64 = torch.float64


def seen(ctx, n, words, window, sinks):
    """For each of n drafted tokens the cached tokens that it sees, ascending.  words: mask words (any
    sign), or None for a chain."""
    rows = []
    for i in range(n):
        drafted = [j for j in range(n) if (j <= i if words is None else (words[i] >> j) & 1)]
        first = max(0, ctx + len(drafted) - window) if window else 0
        rows.append([j for j in range(ctx) if j < sinks or j >= first] + [ctx + j for j in drafted])
    return rows


def attn_row(q, keys, values, scale):
    """Rows q [G, D] over keys, values [m, D] (float64): (out, lse, sum p |v| / sum p, the largest
    |scale| sum |q k_j|).  Only the rows that a NaN or an infinity belongs to are touched by it."""
    if keys.shape[0] == 0:
        z = torch.zeros_like(q)
        return z, torch.full(q.shape[:1], -math.inf, dtype=F64, device=q.device), z, 0.0
    s = scale * (q @ keys.T)
    m = s.max(dim=1, keepdim=True).values
    p = torch.where(s == -math.inf, torch.zeros_like(s), torch.exp(s - m))
    total = p.sum(1, keepdim=True)
    out, mag = p @ values / total, p @ values.abs() / total
    empty = total.squeeze(1) == 0  # every score is -infinity
    out[empty], mag[empty] = 0.0, 0.0
    lse = (m + torch.log(total)).squeeze(1)
    lse = torch.where(m.squeeze(1) == math.inf, m.squeeze(1), lse)
    spread = abs(scale) * float((q.abs() @ keys.abs().T).nan_to_num(0.0, 0.0, 0.0).max())
    return out, lse, mag, spread


def order(x):
    """Indexes of a row of logits from the largest on: NaN above all, equals by index."""
    v = x.to(F64).tolist()
    return sorted(range(len(v)), key=lambda i: (not math.isnan(v[i]), -v[i] if v[i] == v[i] else 0.0, i))


def logprob_row(x, factor):
    """(log probabilities of all tokens, lse, entropy) of one row of logits."""
    nan = torch.full_like(x, math.nan, dtype=F64)
    if not (factor > 0 and math.isfinite(factor)):
        return nan, math.nan, math.nan
    z = x.to(F64) * factor
    if bool(torch.isnan(z).any()):
        return nan, math.nan, math.nan
    m = float(z.max())
    if m == -math.inf:
        return torch.full_like(nan, -math.inf), -math.inf, 0.0
    if m == math.inf:
        return z - math.inf, math.inf, math.nan
    lse = m + math.log(float(torch.exp(z - m).sum()))
    p = torch.exp(z - lse)
    body = torch.where(p > 0, p * (z - lse), torch.zeros_like(p))
    return z - lse, lse, -float(body.sum())


def move(cache, src, dst, starts, page_size):
    """cache [pages, page_size, heads, D] after the groups' moves, one after another."""
    out = cache.clone()
    slots = cache.shape[0] * page_size
    for a, b in zip(starts[:-1], starts[1:]):
        for i in range(a, b):
            if 0 <= src[i] < slots and 0 <= dst[i] < slots:
                out[dst[i] // page_size, dst[i] % page_size] = out[src[i] // page_size, src[i] % page_size].clone()
    return out
