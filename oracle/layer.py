"""The decoder-layer operators of include/decode.h in 64 bits -- TEST INFRASTRUCTURE ONLY.

Plain statements (torch, float64, one sequence and head at a time where that is simplest) of
the RMS norm with its 8-bit outputs, the rotary table and rotation, the cache append and the
attention of one new token over a paged cache.  They run on any device and share no code with
the CUDA library.
"""
from __future__ import annotations

import math

import torch

F64 = torch.float64
E4M3_MAX = 448.0


def rms_norm(x, residual, weight, eps):
    """(h, y) in float64: h = x + residual, y = h / sqrt(mean(h^2) + eps) * weight."""
    h = x.to(F64)
    if residual is not None:
        h = h + residual.to(F64)
    y = h / torch.sqrt((h * h).mean(dim=1, keepdim=True) + eps)
    if weight is not None:
        y = y * weight.to(F64)
    return h, y


def quantize_i8(y):
    """(codes, scales): scale = max |y| / 127 (1 for a zero row), codes rint(y / scale)."""
    scale = y.abs().amax(dim=1) / 127.0
    scale = torch.where(scale > 0, scale, torch.ones_like(scale))
    return torch.round(y / scale[:, None]).clamp(-127, 127), scale


def e4m3_round(v):
    """Float64 -> the nearest E4M3 value (ties to even), saturated to +-448."""
    a = v.abs().clamp(max=E4M3_MAX)
    e = torch.floor(torch.log2(a.clamp(min=2.0 ** -6)))
    e = torch.where(torch.exp2(e) > a.clamp(min=2.0 ** -6), e - 1, e)
    unit = torch.exp2(e - 3)
    return torch.copysign((torch.round(a / unit) * unit).clamp(max=E4M3_MAX), v)


def quantize_mx(y):
    """(values, exponents): per 32 values X = clamp(floor(log2 max |y|) - 8, -127, 127)
    (-127 for a zero block) and the E4M3 values nearest y * 2^-X."""
    M, H = y.shape
    b = y.reshape(M, H // 32, 32)
    most = b.abs().amax(dim=2)
    x = torch.frexp(most).exponent.to(F64) - 1 - 8
    x = torch.where(most > 0, x, torch.full_like(x, -127.0)).clamp(-127, 127)
    return e4m3_round(b * torch.exp2(-x)[:, :, None]).reshape(M, H), x


def rope_frequencies(rot_dim, base, kind="none", factor=1.0, low=0.0, high=1.0,
                     original_len=1.0):
    """f(j) for j < rot_dim / 2, scaled: "none", "linear" (f / factor), "base" (base *
    factor^(rot/(rot-2))), "ramp" (w f + (1 - w) f / factor by the turns over the trained
    length)."""
    out = []
    for j in range(rot_dim // 2):
        b = base * factor ** (rot_dim / (rot_dim - 2)) if kind == "base" else base
        f = b ** (-2.0 * j / rot_dim)
        if kind == "linear":
            f /= factor
        if kind == "ramp":
            turns = original_len * f / (2.0 * math.pi)
            w = min(1.0, max(0.0, (turns - low) / (high - low)))
            f = w * f + (1.0 - w) * f / factor
        out.append(f)
    return torch.tensor(out, dtype=F64)


def rope_table(freq, table_len, magnitude=1.0):
    """[table_len][rot]: cosines, then sines, of position * frequency, in float64."""
    angle = torch.arange(table_len, dtype=F64)[:, None] * freq
    return magnitude * torch.cat([torch.cos(angle), torch.sin(angle)], dim=1)


def rope(x, table_rows, rot_dim, interleaved):
    """x [T, heads, D] turned by table_rows [T, rot]; also |a cos| + |b sin| per value, the
    magnitude its rounding errors scale with."""
    x = x.to(F64)
    half = rot_dim // 2
    y, mag = x.clone(), x.abs().clone()
    for j in range(half):
        i0, i1 = (2 * j, 2 * j + 1) if interleaved else (j, j + half)
        c = table_rows[:, None, j].to(F64)
        s = table_rows[:, None, half + j].to(F64)
        a, b = x[:, :, i0], x[:, :, i1]
        y[:, :, i0] = a * c - b * s
        y[:, :, i1] = b * c + a * s
        mag[:, :, i0] = (a * c).abs() + (b * s).abs()
        mag[:, :, i1] = (b * c).abs() + (a * s).abs()
    return y, mag


def attn(q, keys, values, scale):
    """One query row q [D] over keys, values [n, D] (float64): (out, lse, sum p |v| / sum p,
    max_j |scale| sum |q k_j|)."""
    if keys.shape[0] == 0:
        z = torch.zeros_like(q)
        return z, -math.inf, z, 0.0
    s = scale * (keys @ q)
    m = s.max()
    p = torch.exp(s - m)
    out = (p @ values) / p.sum()
    mag = (p @ values.abs()) / p.sum()
    spread = abs(scale) * float((keys.abs() @ q.abs()).max())
    return out, float(m + torch.log(p.sum())), mag, spread


def cached_tokens(cache, pages, page_size, first, last, head):
    """Tokens first..last-1 of one head from a cache [pages, page_size, heads, D] (float64)."""
    j = torch.arange(first, last, device=cache.device)
    page = pages[j // page_size].long()
    return cache.view(torch.uint8)[page, j % page_size, head].view(cache.dtype).to(F64) \
        if cache.dtype == torch.float8_e4m3fn else cache[page, j % page_size, head].to(F64)
