"""The decoder-layer operators (include/decode.h) at the ends of what their arguments may be."""
import math

import pytest
import torch

import weight_only_int4_tma_gb300 as w4
from oracle import layer as od

pytestmark = pytest.mark.gpu

F64 = torch.float64
E4M3 = torch.float8_e4m3fn
U = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
CODE = {torch.float16: w4.W4A16_FP16, torch.bfloat16: w4.W4A16_BF16}
DTYPES = [torch.float16, torch.bfloat16]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from weight_only_int4_tma_gb300 import build
    build.build()


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(shape, dtype, seed, scale=1.0):
    return (torch.randn(shape, generator=_gen(seed), device="cuda") * scale).to(dtype)


def _close(out, q, K, V, dtype):
    """One row of attention against the statement: a score is a sum of D products, weights are carried
    to 2^-15, one addition of 2^-23 per token, exp and the joins 2^-21."""
    want, _, mag, spread = od.attn(q.to(F64), K.to(F64), V.to(F64), len(q) ** -0.5)
    eps = 2 * spread * (len(q) + 8) * 2.0 ** -23 + 2.0 ** -15 + len(K) * 2.0 ** -23 + 2.0 ** -21
    assert bool(((out.to(F64) - want).abs() <= want.abs() * U[dtype] + 2 * eps * mag + 2.0 ** -25).all())


@pytest.mark.parametrize("page_size", [0x7FFF0000, 1 << 30])
def test_one_page_of_any_size(page_size):
    """A flat cache told as one page of up to 2^31 slots, of which the first hundred are there."""
    n, h, D, dtype = 100, 2, 64, torch.float16
    k, v = (torch.zeros(n, h, D, dtype=dtype, device="cuda") for _ in range(2))
    cache = w4.KvCache(k.data_ptr(), v.data_ptr(), None, None, 0, h * D, D, 0, h * D, D, 1, page_size, h, D,
                       w4.DEC_KV_FP16, 0)
    new_k, new_v, q = (_randn((n, h * D), dtype, s) for s in range(3))
    rc = w4.rope_config(0, h, D, CODE[dtype], None, 0)
    w4.dec_rope_append(rc, cache, None, new_k, new_v, n, torch.zeros(n, dtype=torch.int32, device="cuda"),
                       torch.arange(n, device="cuda"), None)
    assert w4.w4a16_get_device_status() == 0
    assert torch.equal(k.view(n, -1), new_k) and torch.equal(v.view(n, -1), new_v)
    cfg = w4.attn_config(h, CODE[dtype], D ** -0.5, 1)
    out = torch.empty(1, h * D, dtype=dtype, device="cuda")
    w4.dec_attn_paged(cfg, cache, q[:1], torch.zeros(1, 1, dtype=torch.int32, device="cuda"),
                      torch.tensor([n], dtype=torch.int32, device="cuda"), 1, out, None, w4.attn_workspace(cfg, cache))
    assert w4.w4a16_get_device_status() == 0
    for i in range(h):
        row = slice(i * D, (i + 1) * D)
        _close(out[0, row], q[0, row], k[:, i], v[:, i], dtype)


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("M,H", [(3, 128), (5, 4096), (200, 1152)])
def test_a_zero_row_without_eps(M, H, dtype):
    """eps = 0: int8 and MX write a zero row as zeros (scale 1, exponent byte 0), and its neighbours as
    without it; the 16-bit form is 0 / 0."""
    x = _randn((M, H), dtype, H)
    x[M // 2] = 0
    rows = [m for m in range(M) if m != M // 2]
    codes, s = torch.empty(M, H, dtype=torch.int8, device="cuda"), torch.empty(M, device="cuda")
    w4.dec_rms_norm_i8(x, None, None, M, H, CODE[dtype], 0.0, None, codes, s)
    assert bool((codes[M // 2] == 0).all()) and float(s[M // 2]) == 1.0
    _, y = od.rms_norm(x[rows], None, None, 0.0)
    want, scale = od.quantize_i8(y)
    # sums of at most 2^8 roundings, halved by the root, and products: 2^-16
    assert bool(((s[rows].to(F64) - scale).abs() <= scale * 2.0 ** -15).all())
    assert bool(((codes[rows].to(F64) - y / scale[:, None]).abs() <= 0.5 + 127 * 2.0 ** -14).all())
    codes, s = torch.empty(M, H, dtype=torch.uint8, device="cuda"), torch.empty(M, H // 32, dtype=torch.uint8, device="cuda")
    w4.dec_rms_norm_mx(x, None, None, M, H, CODE[dtype], 0.0, None, codes, s)
    assert bool((codes[M // 2] == 0).all()) and bool((s[M // 2] == 0).all())
    assert not bool((codes[rows] & 0x7F == 0x7F).any())
    out = torch.empty_like(x)
    w4.dec_rms_norm(x, None, None, M, H, CODE[dtype], 0.0, None, out)
    assert bool(out[M // 2].isnan().all()) and bool(out[rows].isfinite().all())
    assert w4.w4a16_get_device_status() == 0


@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("M,H", [(3, 128), (5, 4096), (200, 1152), (2, 32768)])
def test_int8_scale_of_a_row_with_infinities_or_nan(M, H, dtype, value):
    """The scale is NaN, so that what is computed from the row is; its neighbours do not change."""
    x = _randn((M, H), dtype, H + M)
    codes, s = torch.empty(M, H, dtype=torch.int8, device="cuda"), torch.empty(M, device="cuda")
    w4.dec_rms_norm_i8(x, None, None, M, H, CODE[dtype], 1e-5, None, codes, s)
    want = codes.clone(), s.clone()
    x[M - 1, H // 3] = value
    w4.dec_rms_norm_i8(x, None, None, M, H, CODE[dtype], 1e-5, None, codes, s)
    assert w4.w4a16_get_device_status() == 0
    assert math.isnan(float(s[M - 1]))
    assert torch.equal(codes[:-1], want[0][:-1]) and torch.equal(s[:-1], want[1][:-1])


@pytest.mark.parametrize("D,rot", [(128, 128), (16, 6)])  # both kernels
def test_append_by_scales_of_any_size(D, rot):
    """8-bit values are the nearest to the fp32 quotient for scales down to the smallest subnormal number
    and up to the largest; zeros stay zeros."""
    scales = [2.0 ** -149, 1e-39, 2.0 ** -128, 2.0 ** -126, 2.0 ** -100, 3e-25, 0.05, 1e24, 1e30, 3e38, math.inf]
    h, T, page, dtype = len(scales), 512, 16, torch.bfloat16
    s = torch.tensor(scales, device="cuda")
    x = torch.randn(T, h, D, generator=_gen(1), device="cuda") * 8
    x = (x.double() * s.double().clamp(max=3e35)[:, None]).float().to(dtype)  # subnormal numbers among them
    x[:, :, 0], x[:, :, 1] = 0.0, -0.0
    x[:, :, 2], x[:, :, 3], x[:, :, 4] = math.inf, 3e38, -1e-38
    table = torch.zeros(1, rot, device="cuda")
    table[:, :rot // 2] = 1  # turned by nothing
    kc, vc = (torch.zeros(T // page, page, h, D, device="cuda").to(E4M3) for _ in range(2))
    cfg = w4.rope_config(0, h, D, CODE[dtype], table, rot, w4.DEC_ROPE_INTERLEAVED)
    rows = x.view(T, h * D)
    w4.dec_rope_append(cfg, w4.kv_cache(kc, vc, s, s), None, rows, rows, T,
                       torch.zeros(T, dtype=torch.int32, device="cuda"), torch.arange(T, device="cuda"), None)
    assert w4.w4a16_get_device_status() == 0
    value = x.cpu().float()
    a, b = value[..., 0:rot:2], value[..., 1:rot:2]  # the turn itself loses zeros' signs, and infinities
    turned = torch.stack([a * 1.0 - b * 0.0, b * 1.0 + a * 0.0], -1).flatten(-2)
    for c, v in ((vc, value), (kc, torch.cat([turned, value[..., rot:]], -1))):
        want = (v / s.cpu()[:, None]).clamp(-448, 448).to(E4M3).view(torch.uint8)
        got = c.view(torch.uint8).view(T, h, D).cpu()
        nan = want & 0x7F == 0x7F
        assert bool((got[nan] & 0x7F == 0x7F).all())
        assert torch.equal(got[~nan], want[~nan]), ((got != want) & ~nan).sum((0, 2))


def test_as_many_rows_and_tokens_as_an_int_counts():
    """2^31 - 1 rows of 8 values, normed and turned in place."""
    M, dtype = 0x7FFFFFFF, torch.bfloat16
    if torch.cuda.mem_get_info()[0] < (64 << 30):
        pytest.skip("not enough memory")
    x = torch.full((M, 8), 2.0, dtype=dtype, device="cuda")  # 32 GiB
    w4.dec_rms_norm(x, None, None, M, 8, CODE[dtype], 0.0, None, x)
    assert w4.w4a16_get_device_status() == 0
    for part in x.view(-1).split(1 << 31):
        assert bool((part == 1).all())
    positions = torch.zeros(M, dtype=torch.int32, device="cuda")
    table = torch.tensor([[0.0] * 4 + [1.0] * 4], device="cuda")  # a quarter turn
    x[:, :4] = 3
    w4.dec_rope_append(w4.rope_config(1, 0, 8, CODE[dtype], table, 8), None, x, None, None, M, positions, None, x)
    assert w4.w4a16_get_device_status() == 0
    for part in x.split(1 << 28):
        assert bool((part[:, :4] == -1).all()) and bool((part[:, 4:] == 3).all())


@pytest.mark.parametrize("B", [3 << 17, (5 << 21) + 5])
def test_attention_of_millions_of_sequences(B):
    """One token each, every ninth sequence empty: the output is the token's value."""
    D, pages, dtype = 8, 4096, torch.bfloat16
    kc, vc = (_randn((pages, 1, 1, D), dtype, s) for s in range(2))
    q = torch.full((B, D), 0.5, dtype=dtype, device="cuda")
    table = torch.randint(0, pages, (B, 1), generator=_gen(2), device="cuda").int()
    lens = (torch.arange(B, device="cuda") % 9 != 8).int()
    cfg, cache = w4.attn_config(1, CODE[dtype], 1.0, 1), w4.kv_cache(kc, vc)
    out = torch.full((B, D), 7.0, dtype=dtype, device="cuda")
    w4.dec_attn_paged(cfg, cache, q, table, lens, B, out, None, w4.attn_workspace(cfg, cache))
    assert w4.w4a16_get_device_status() == 0
    assert torch.equal(out, vc.view(pages, D)[table[:, 0].long()] * lens[:, None].to(dtype))
