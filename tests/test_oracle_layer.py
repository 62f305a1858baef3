"""The 64-bit statements of the decoder-layer operators, pinned by closed forms and by torch's
own float8 conversion (CPU)."""
import math

import pytest
import torch

from oracle import layer as od

F64 = torch.float64


def test_norm_of_constant_row_is_weight():
    w = torch.tensor([1.0, -2.0, 0.5, 4.0])
    h, y = od.rms_norm(torch.full((1, 4), 3.0), torch.full((1, 4), 2.0), w, 0.0)
    assert torch.equal(h, torch.full((1, 4), 5.0, dtype=F64))
    assert torch.allclose(y[0], w.to(F64), rtol=1e-15, atol=0)


def test_norm_zero_row_needs_eps():
    _, y = od.rms_norm(torch.zeros(1, 8), None, None, 1e-6)
    assert torch.equal(y, torch.zeros(1, 8, dtype=F64))


def test_quantize_i8_ties_zero_rows_and_range():
    y = torch.tensor([[127.0, 0.5, 1.5, -2.5], [0.0, 0.0, 0.0, 0.0]], dtype=F64)
    q, s = od.quantize_i8(y)
    assert q.tolist() == [[127, 0, 2, -2], [0, 0, 0, 0]] and s.tolist() == [1.0, 1.0]


def test_e4m3_round_equals_torch_on_every_code_and_midpoint():
    codes = torch.arange(0, 127, dtype=torch.uint8).view(torch.float8_e4m3fn).to(torch.float32)
    mid = (codes[1:] + codes[:-1]) / 2
    v = torch.cat([codes, mid, mid * (1 + 2.0 ** -20), mid * (1 - 2.0 ** -20)])
    v = torch.cat([v, -v])
    want = v.to(torch.float8_e4m3fn).to(F64)
    assert torch.equal(od.e4m3_round(v.to(F64)), want)
    assert od.e4m3_round(torch.tensor([1e9, -500.0], dtype=F64)).tolist() == [448.0, -448.0]


@pytest.mark.parametrize("most,x", [(448.0, 0), (256.0, 0), (255.0, -1), (1.0, -8), (0.0, -127),
                                    (2.0 ** -125, -127), (2.0 ** 100, 92)])
def test_quantize_mx_exponent(most, x):
    y = torch.zeros(1, 32, dtype=F64)
    y[0, 7] = most
    v, e = od.quantize_mx(y)
    assert e.tolist() == [[x]]
    assert float(v[0, 7]) == float(od.e4m3_round(torch.tensor(most * 2.0 ** -x, dtype=F64)))


def test_quantize_mx_matches_the_format_oracle():
    import numpy as np
    from oracle import mxfp
    y = torch.from_numpy(np.random.default_rng(0).standard_normal((2, 96)) * 5)
    v, e = od.quantize_mx(y)
    codes, exps = mxfp.quantize_mx(y.numpy(), mxfp.E4M3)
    assert np.array_equal(e.numpy() + 127, exps)
    assert np.array_equal(v.numpy(), mxfp._values(mxfp.E4M3)[codes])


def test_rope_turns_by_the_angle():
    f = od.rope_frequencies(4, 100.0)
    assert torch.allclose(f, torch.tensor([1.0, 0.1], dtype=F64), rtol=1e-15)
    t = od.rope_table(f, 3)
    x = torch.tensor([[[1.0, 1.0, 0.0, 0.0, 7.0]]])
    y, _ = od.rope(x, t[2:3], 4, False)
    want = [math.cos(2), math.cos(0.2), math.sin(2), math.sin(0.2), 7.0]
    assert torch.allclose(y[0, 0], torch.tensor(want, dtype=F64), rtol=1e-14)
    y, _ = od.rope(torch.tensor([[[1.0, 0.0, 1.0, 0.0, 7.0]]]), t[2:3], 4, True)
    want = [math.cos(2), math.sin(2), math.cos(0.2), math.sin(0.2), 7.0]
    assert torch.allclose(y[0, 0], torch.tensor(want, dtype=F64), rtol=1e-14)


def test_rope_keeps_relative_positions():
    """q . k after the turn depends on the positions' difference alone."""
    g = torch.Generator().manual_seed(1)
    q, k = (torch.randn(1, 1, 64, generator=g, dtype=F64) for _ in range(2))
    t = od.rope_table(od.rope_frequencies(64, 10000.0), 200)
    dots = [float((od.rope(q, t[p:p + 1], 64, False)[0] * od.rope(k, t[p - 5:p - 4], 64, False)[0]).sum())
            for p in (5, 77, 199)]
    assert max(dots) - min(dots) < 1e-12


def test_rope_scalings():
    plain = od.rope_frequencies(64, 10000.0)
    assert torch.allclose(od.rope_frequencies(64, 10000.0, "linear", 4.0), plain / 4)
    b = od.rope_frequencies(64, 10000.0, "base", 4.0)
    assert float(b[0]) == 1.0 and math.isclose(float(b[-1]), float(plain[-1]) / 4, rel_tol=1e-12)
    r = od.rope_frequencies(64, 10000.0, "ramp", 4.0, low=1.0, high=32.0, original_len=2048.0)
    assert float(r[0]) == 1.0 and math.isclose(float(r[-1]), float(plain[-1]) / 4, rel_tol=1e-12)
    assert bool(((r <= plain) & (r >= plain / 4 - 1e-18)).all())


def test_attn_closed_forms():
    k = torch.zeros(3, 4, dtype=F64)
    v = torch.arange(12, dtype=F64).view(3, 4)
    q = torch.ones(4, dtype=F64)
    out, lse, _, _ = od.attn(q, k, v, 0.5)
    assert torch.allclose(out, v.mean(0)) and math.isclose(lse, math.log(3))
    out, lse, _, _ = od.attn(q, k[:0], v[:0], 0.5)
    assert torch.equal(out, torch.zeros(4, dtype=F64)) and lse == -math.inf
    k[1] = 1000.0
    out, lse, _, _ = od.attn(q, k, v, 0.5)
    assert torch.equal(out, v[1]) and lse == 2000.0


def test_cached_tokens_follow_the_block_table():
    cache = torch.arange(4 * 3 * 2 * 2, dtype=torch.float32).view(4, 3, 2, 2)
    got = od.cached_tokens(cache, torch.tensor([2, 0, 3]), 3, 2, 5, 1)
    want = torch.stack([cache[2, 2, 1], cache[0, 0, 1], cache[0, 1, 1]]).to(F64)
    assert torch.equal(got, want)
