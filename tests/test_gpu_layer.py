"""GPU parity of the decoder-layer operators (include/decode.h) against their 64-bit statements
(oracle/layer.py).

Tolerances, from the operations that round:
  U       one rounding to the stored type: 2^-8 (bf16), 2^-11 (fp16) of the value, and half of
          fp16's smallest step, 2^-25.
  norm    sums of at most 2^15 squares per row in fp32, each thread adding at most 2^7 of them in
          order and a tree above: below 2^8 roundings of 2^-24, halved by the square root, plus
          a few for the products: NORM = 2^-16 relative.
  rope    two products and a sum: 3 roundings of 2^-24 of |a cos| + |b sin|: ROPE = 2^-22.
  attn    a score is a sum of D products: ds = (D + 8) 2^-23 max_j scale sum |q k|, which moves a
          weight by ds relative, twice (numerator and denominator); weights carried to 2^-15
          relative; len additions of 2^-23 at most; exp and the join 2^-21.
"""
import math

import pytest
import torch

import weight_only_int4_tma_gb300 as w4
from oracle import layer as od

pytestmark = pytest.mark.gpu

F64 = torch.float64
U = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float16: 2.0 ** -25, torch.bfloat16: 0.0}
CODE = {torch.float16: w4.W4A16_FP16, torch.bfloat16: w4.W4A16_BF16}
E4M3 = torch.float8_e4m3fn
NORM, ROPE = 2.0 ** -16, 2.0 ** -22
DTYPES = [torch.float16, torch.bfloat16]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from weight_only_int4_tma_gb300 import build
    build.build()


def _status():
    return w4.w4a16_get_device_status()


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(shape, dtype, g, scale=1.0):
    x = torch.randn(shape, generator=g, device="cuda") * scale
    return x.to(dtype)


def _within(got, want, tol, what):
    """|got - want| <= tol everywhere (float64 tensors)."""
    off = (got.to(F64) - want).abs()
    bad = ~(off <= tol)
    assert not bool(bad.any()), (f"{what}: {int(bad.sum())} of {bad.numel()} outside; worst "
                                 f"{float((off / tol.clamp(min=1e-300)).max()):.3g} x the bound")


def _e4m3_tol(z):
    """Half of E4M3's step around z (saturated values are exact)."""
    a = z.abs().clamp(min=2.0 ** -6, max=448.0)
    return torch.exp2(torch.floor(torch.log2(a)) - 4)


# ---- norm -------------------------------------------------------------------------------------

NORM_SHAPES = [(1, 8), (1, 1), (3, 7), (2, 130), (5, 1000), (7, 4096), (1, 8192), (2, 8200),
               (33, 4097), (300, 512), (4, 16384), (2, 32768), (1, 40000), (1500, 64)]


def _norm_inputs(M, H, dtype, seed, residual=True, ldx=0, ldr=0, offset=0):
    g = _gen(seed)

    def rows(ld, scale):
        full = _randn(M * (ld or H) + 8, dtype, g, scale)
        return full[offset:].as_strided((M, H), (ld or H, 1))
    x = rows(ldx, 1.0)
    r = rows(ldr, 3.0) if residual else None
    w = _randn(H + 8, dtype, g, 0.2)[offset:offset + H] + 1
    return x, r, w


def _check_norm(x, r, w, dtype, y, rout, eps):
    h, want = od.rms_norm(x, r, w, eps)
    _within(y, want, want.abs() * (U[dtype] + NORM) + TINY[dtype], "y")
    if rout is not None:
        # x + residual is one fp32 addition before the rounding
        _within(rout, h, h.abs() * (U[dtype] + 2.0 ** -23) + TINY[dtype], "residual_out")


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("M,H", NORM_SHAPES)
def test_norm(M, H, dtype):
    x, r, w = _norm_inputs(M, H, dtype, M + H)
    y, rout = torch.empty(M, H, dtype=dtype, device="cuda"), torch.empty(M, H, dtype=dtype, device="cuda")
    w4.dec_rms_norm(x, r, w, M, H, CODE[dtype], 1e-5, rout, y)
    assert _status() == 0
    _check_norm(x, r, w, dtype, y, rout, 1e-5)


@pytest.mark.parametrize("H,ldx,ldr,ldy,offset", [(64, 72, 80, 88, 0), (64, 67, 71, 65, 0),
                                                  (512, 512, 1024, 520, 3), (100, 104, 100, 112, 1)])
def test_norm_strides_and_alignment(H, ldx, ldr, ldy, offset):
    M, dtype = 9, torch.bfloat16
    x, r, w = _norm_inputs(M, H, dtype, H + ldx, ldx=ldx, ldr=ldr, offset=offset)
    ybuf = torch.full((M, ldy), 7.0, dtype=dtype, device="cuda")
    rbuf = torch.full((M * ldr + 8,), 7.0, dtype=dtype, device="cuda")
    w4.dec_rms_norm(x, r, w, M, H, CODE[dtype], 1e-6, rbuf[offset:], ybuf, ldx=ldx, ldr=ldr, ldy=ldy)
    assert _status() == 0
    _check_norm(x, r, w, dtype, ybuf[:, :H], rbuf[offset:].as_strided((M, H), (ldr, 1)), 1e-6)
    assert bool((ybuf[:, H:] == 7).all())  # nothing between the rows
    gaps = torch.ones(M * ldr + 8, dtype=torch.bool, device="cuda")
    gaps[offset:].as_strided((M, H), (ldr, 1)).fill_(False)
    assert bool((rbuf[gaps] == 7).all())


@pytest.mark.parametrize("H", [512, 515, 8192])
def test_norm_in_place_and_optional_arguments(H):
    M, dtype = 5, torch.float16
    x, r, w = _norm_inputs(M, H, dtype, H)
    x, r = x.contiguous(), r.contiguous()
    y, rout = x.clone(), r.clone()
    w4.dec_rms_norm(y, rout, w, M, H, CODE[dtype], 1e-5, rout, y)
    _check_norm(x, r, w, dtype, y, rout, 1e-5)
    w4.dec_rms_norm(x, None, None, M, H, CODE[dtype], 0.0, None, y)
    _check_norm(x, None, None, dtype, y, None, 0.0)
    w4.dec_rms_norm(x, r, w, M, H, CODE[dtype], 1e-5, None, y)
    _check_norm(x, r, w, dtype, y, None, 1e-5)
    assert _status() == 0


@pytest.mark.parametrize("H", [64, 77, 4096])
def test_norm_extreme_rows(H):
    """Zero rows, rows at the ends of the range, and a NaN that stays in its row."""
    dtype = torch.bfloat16
    x = torch.randn(5, H, device="cuda", generator=_gen(1)).to(dtype)
    x[0] = 0
    x[1] = x[1] * 1e15
    x[2] = x[2] * 1e-25
    x[3, H // 2] = math.nan
    y = torch.empty_like(x)
    w4.dec_rms_norm(x, None, None, 5, H, CODE[dtype], 1e-6, None, y)
    assert _status() == 0
    assert bool((y[0] == 0).all()) and bool(y[3].isnan().all())
    keep = [0, 1, 2, 4]
    _check_norm(x[keep], None, None, dtype, y[keep], None, 1e-6)


Q_SHAPES = [(1, 128), (3, 64), (8, 8192), (5, 1152), (37, 4096), (2, 32768), (400, 256), (2, 2080)]


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("M,H", Q_SHAPES)
def test_norm_i8(M, H, dtype):
    x, r, w = _norm_inputs(M, H, dtype, 3 * M + H)
    if M > 1:
        x[M - 1], r[M - 1] = 0, 0
    codes = torch.empty(M, H, dtype=torch.int8, device="cuda")
    s = torch.empty(M, device="cuda")
    rout = torch.empty(M, H, dtype=dtype, device="cuda")
    w4.dec_rms_norm_i8(x, r, w, M, H, CODE[dtype], 1e-5, rout, codes, s)
    assert _status() == 0
    h, y = od.rms_norm(x, r, w, 1e-5)
    _, scale = od.quantize_i8(y)
    _within(s, scale, scale * 2 * NORM, "s_y")
    _within(codes, y / scale[:, None], torch.full_like(y, 0.5 + 127 * 4 * NORM), "codes")
    assert int(codes.abs().max()) <= 127
    _within(rout, h, h.abs() * (U[dtype] + 2.0 ** -23) + TINY[dtype], "residual_out")


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("M,H", Q_SHAPES)
def test_norm_mx(M, H, dtype):
    x, r, w = _norm_inputs(M, H, dtype, 5 * M + H)
    x[0, :32], r[0, :32] = 0, 0  # a zero block
    codes = torch.empty(M, H, dtype=torch.uint8, device="cuda")
    s = torch.empty(M, H // 32, dtype=torch.uint8, device="cuda")
    rout = torch.empty(M, H, dtype=dtype, device="cuda")
    w4.dec_rms_norm_mx(x, r, w, M, H, CODE[dtype], 1e-5, rout, codes, s)
    assert _status() == 0
    h, y = od.rms_norm(x, r, w, 1e-5)
    # the exponent may only differ where the block's largest value is at a power of two
    lo, hi = od.quantize_mx(y * (1 - 2 * NORM))[1], od.quantize_mx(y * (1 + 2 * NORM))[1]
    e = s.to(F64) - 127
    assert bool(((e == lo) | (e == hi)).all())
    z = (y.view(M, -1, 32) * torch.exp2(-e)[:, :, None]).view(M, H)
    z = z.clamp(-448, 448)
    _within(codes.view(E4M3).to(F64), z, _e4m3_tol(z) + z.abs() * 2 * NORM, "codes")
    assert int(s[0, 0]) == 0 and bool((codes[0, :32] == 0).all())
    _within(rout, h, h.abs() * (U[dtype] + 2.0 ** -23) + TINY[dtype], "residual_out")


@pytest.mark.parametrize("scale", [1e-19, 1e-17])
def test_norm_i8_tiny_rows(scale):
    """Rows whose 127 / max |y| passes fp32's range: the codes are as of any other row."""
    M, H, dtype = 3, 512, torch.bfloat16
    x, _, w = _norm_inputs(M, H, dtype, 17, residual=False)
    w = (w.double() * scale).to(dtype)
    x = (x.double() * 1e-18).to(dtype)  # eps decides: y = h * weight
    codes, s = torch.empty(M, H, dtype=torch.int8, device="cuda"), torch.empty(M, device="cuda")
    w4.dec_rms_norm_i8(x, None, w, M, H, CODE[dtype], 1.0, None, codes, s)
    assert _status() == 0
    _, y = od.rms_norm(x, None, w, 1.0)
    _, want = od.quantize_i8(y)
    assert float(want.max()) < 1e-33
    # the products round to normal numbers down to 2^-126 and in steps of 2^-149 below
    _within(s, want, want * 2 * NORM + 2.0 ** -149, "s_y")
    _within(codes, y / want[:, None], 0.5 + 127 * 4 * NORM + 2.0 ** -149 / want[:, None].expand_as(y), "codes")


def test_norm_feeds_the_w4a8_and_mx_gemms():
    """The 8-bit rows are what the GEMMs take: the product with the quantised rows themselves."""
    import numpy as np
    import oracle
    import synth_inputs as si
    from oracle import w4a8 as o8
    M, N, K, dtype = 5, 96, 512, torch.float16
    x, r, w = _norm_inputs(M, K, dtype, 11)
    codes, s = torch.empty(M, K, dtype=torch.int8, device="cuda"), torch.empty(M, device="cuda")
    w4.dec_rms_norm_i8(x, r, w, M, K, CODE[dtype], 1e-5, None, codes, s)
    c = si.make_w4a8_case(M, N, K, dtype=si.FP16, seed=2)
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    packed = torch.empty(w4.w4a8_packed_bytes(N, K), dtype=torch.uint8, device="cuda")
    w4.w4a8_repack(dev(c.qweight.view(np.int32)), dev(c.s_u8), dev(c.a), dev(c.s_w), N, K, packed)
    Y = torch.empty(M, N, dtype=torch.int16, device="cuda")
    w4.w4a8_gemm(codes, s, packed, M, N, K, si.FP16, Y)
    assert _status() == 0
    want = o8.gemm_codes(codes.cpu().numpy().astype(np.int64), s.cpu().numpy(), c.qweight, c.s_u8,
                         c.a, c.s_w, N, K)
    assert np.array_equal(Y.cpu().numpy().view(np.uint16), oracle.encode(want.astype(np.float64), si.FP16))


# ---- rotary positions and the append --------------------------------------------------------------

@pytest.mark.parametrize("kind,args", [("none", {}), ("linear", dict(factor=4.0)),
                                       ("base", dict(factor=8.0)),
                                       ("ramp", dict(factor=8.0, low=1.0, high=32.0, original_len=4096.0))])
@pytest.mark.parametrize("rot", [4, 64, 128])
def test_rope_table(rot, kind, args):
    n, magnitude = 20011, 1.25
    kinds = {"none": 0, "linear": 1, "base": 2, "ramp": 3}
    s = w4.RopeScaling(kinds[kind], args.get("factor", 1), args.get("low", 0), args.get("high", 1),
                       args.get("original_len", 1), magnitude)
    table = torch.empty(n, rot, device="cuda")
    w4.dec_rope_table(rot, 500000.0, s, table, n)
    assert _status() == 0
    want = od.rope_table(od.rope_frequencies(rot, 500000.0, kind, **args), n, magnitude)
    # fp64 angles up to 2^15 (2^-37 of rounding), then one rounding to fp32
    _within(table.cpu(), want, want.abs() * 2.0 ** -24 + 2.0 ** -36, "table")


def _cache_tensors(pages, size, heads, D, kv, g, hnd=False, fill=1.0):
    shape = (pages, heads, size, D) if hnd else (pages, size, heads, D)
    x = [_randn(shape, torch.float16 if kv == E4M3 else kv, g, fill).to(kv) for _ in range(2)]
    return [t.transpose(1, 2) for t in x] if hnd else x


ROPE_CASES = [
    # T, q_heads, kv_heads, D, rot, interleaved, kv, page, hnd
    (1, 64, 8, 128, 128, False, None, 64, False), (7, 8, 8, 64, 64, True, None, 16, True),
    (33, 4, 1, 80, 40, False, None, 8, False), (5, 6, 2, 96, 96, False, E4M3, 16, False),
    (129, 32, 4, 128, 64, True, E4M3, 5, True), (3, 2, 2, 256, 256, False, None, 128, False),
    (2, 3, 3, 8, 2, False, None, 1, False), (4, 5, 5, 16, 6, True, E4M3, 3, False),
    (9, 7, 1, 72, 0, False, None, 16, False), (700, 12, 2, 112, 56, False, None, 32, False),
    (17, 8, 2, 128, 20, False, E4M3, 16, False), (600, 64, 8, 128, 128, True, None, 64, False)]


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("T,hq,hkv,D,rot,inter,kv,page,hnd", ROPE_CASES)
def test_rope_append(T, hq, hkv, D, rot, inter, kv, page, hnd, dtype):
    g = _gen(T + D)
    kv = kv or dtype
    count = -(-T // page) + 3
    table = od.rope_table(od.rope_frequencies(max(rot, 2), 10000.0), 5000).float().cuda()[:, :rot].contiguous()
    qkv = _randn((T, (hq + 2 * hkv) * D + 8), dtype, g)  # rows of a wider projection
    parts = [qkv[:, :hq * D], qkv[:, hq * D:(hq + hkv) * D], qkv[:, (hq + hkv) * D:(hq + 2 * hkv) * D]]
    ld = qkv.stride(0)
    kc, vc = _cache_tensors(count, page, hkv, D, kv, g, hnd)
    before = [c.clone() for c in (kc, vc)]
    scales = [0.05 + 0.1 * torch.rand(hkv, device="cuda", generator=g) if kv == E4M3 else None for _ in range(2)]
    positions = torch.randint(0, 5000, (T,), generator=g, device="cuda").int()
    slots = torch.randperm(count * page, generator=g, device="cuda")[:T]
    if T > 2:
        slots[1] = -1  # a token that is not cached
    cache = w4.kv_cache(kc, vc, *scales)
    cfg = w4.rope_config(hq, hkv, D, CODE[dtype], table if rot else None, rot, int(inter),
                         ldq=ld, ldk=ld, ldv=ld, ldqo=hq * D + 16)
    qo = torch.full((T, hq * D + 16), 3.0, dtype=dtype, device="cuda")
    ko = torch.empty((T, hkv * D), dtype=dtype, device="cuda")
    w4.dec_rope_append(cfg, cache, *parts, T, positions, slots, qo, ko)
    assert _status() == 0
    rows = table[positions.long()]
    for x, got, heads in ((parts[0], qo[:, :hq * D], hq), (parts[1], ko, hkv)):
        want, mag = od.rope(x.reshape(T, heads, D), rows, rot, inter)
        _within(got.reshape(T, heads, D), want, want.abs() * U[dtype] + mag * ROPE * 2 + TINY[dtype], "rotated")
    assert bool((qo[:, hq * D:] == 3).all())
    kept = slots >= 0
    for i, (c, x) in enumerate(((kc, parts[1]), (vc, parts[2]))):
        want, mag = od.rope(x.reshape(T, hkv, D), rows, rot if i == 0 else 0, inter)
        at = slots[kept]
        bits = torch.uint8 if kv == E4M3 else torch.int16
        got = c.view(bits)[at // page, at % page].view(kv).to(F64)
        if kv == E4M3:
            z, m = want / scales[i].to(F64)[:, None], mag / scales[i].to(F64)[:, None]
            z = z.clamp(-448, 448)
            _within(got, z[kept], (_e4m3_tol(z) + m * ROPE * 2)[kept], "cache")
        else:
            _within(got, want[kept], (want.abs() * U[dtype] + mag * ROPE * 2 + TINY[dtype])[kept], "cache")
        untouched = torch.ones(count * page, dtype=torch.bool, device="cuda")
        untouched[at] = False
        u = untouched.nonzero().squeeze(1)
        assert torch.equal(c.view(bits)[u // page, u % page], before[i].view(bits)[u // page, u % page])


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("D,rot", [(128, 128), (64, 20), (80, 40)])
def test_rope_in_place_without_cache(D, rot, inter):
    T, hq, hkv, dtype = 11, 6, 3, torch.bfloat16
    g = _gen(D + rot)
    table = od.rope_table(od.rope_frequencies(rot, 10000.0), 300).float().cuda()
    q, k = _randn((T, hq * D), dtype, g), _randn((T, hkv * D), dtype, g)
    q0, k0 = q.clone(), k.clone()
    positions = torch.arange(T, device="cuda").int() * 7
    cfg = w4.rope_config(hq, hkv, D, CODE[dtype], table, rot, int(inter))
    w4.dec_rope_append(cfg, None, q, k, None, T, positions, None, q, k)
    assert _status() == 0
    for x0, x, heads in ((q0, q, hq), (k0, k, hkv)):
        want, mag = od.rope(x0.view(T, heads, D), table[positions.long()], rot, inter)
        _within(x.view(T, heads, D), want, want.abs() * U[dtype] + mag * ROPE * 2, "rotated")


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
def test_append_rounds_the_quotient_to_nearest(dtype):
    """8-bit values are the nearest to the fp32 quotient, bit for bit; infinities saturate."""
    T, h, D, page = 2048, 8, 128, 16
    g = _gen(3)
    k, v = (_randn((T, h * D), dtype, g, 8.0) for _ in range(2))
    special = torch.tensor([math.inf, -math.inf, 65504.0, -65504.0, 0.0, -0.0, 2.0 ** -24, math.nan], device="cuda")
    k[0, :8], v[5, -8:] = special.to(dtype), special.to(dtype)
    kc, vc = _cache_tensors(T // page, page, h, D, E4M3, g)
    ks, vs = (0.02 + torch.rand(h, device="cuda", generator=g) for _ in range(2))
    cfg = w4.rope_config(0, h, D, CODE[dtype], None, 0)
    w4.dec_rope_append(cfg, w4.kv_cache(kc, vc, ks, vs), None, k, v, T,
                       torch.zeros(T, dtype=torch.int32, device="cuda"), torch.arange(T, device="cuda"), None)
    assert _status() == 0
    for c, x, scale in ((kc, k, ks), (vc, v, vs)):
        want = (x.float().view(T, h, D) / scale[:, None]).clamp(-448, 448).to(E4M3).view(torch.uint8)
        got = c.view(torch.uint8).view(T, h, D)
        nan = x.view(T, h, D).isnan()
        assert torch.equal(got[~nan], want[~nan])
        assert bool((got[nan] & 0x7F == 0x7F).all())


def test_rope_bad_positions_and_slots_are_reported_and_skipped():
    T, h, D, dtype = 4, 2, 64, torch.float16
    g = _gen(0)
    table = od.rope_table(od.rope_frequencies(D, 10000.0), 100).float().cuda()
    q, k, v = (_randn((T, h * D), dtype, g) for _ in range(3))
    cfg = w4.rope_config(h, h, D, CODE[dtype], table, D)
    for positions, slots, wrote in (([0, 100, -1, 5], [0, 1, 2, 3], {0, 3}),
                                    ([0, 1, 2, 3], [0, 32, 1 << 40, 3], {0, 3})):
        kc, vc = (torch.zeros(4, 8, h, D, dtype=dtype, device="cuda") for _ in range(2))
        out = torch.zeros_like(q)
        w4.dec_rope_append(cfg, w4.kv_cache(kc, vc), q, k, v, T,
                           torch.tensor(positions, dtype=torch.int32, device="cuda"),
                           torch.tensor(slots, device="cuda"), out)
        assert _status() == w4.W4A16_ERR_INVALID_ARG
        full = kc.view(-1, h * D).abs().sum(1).nonzero().squeeze(1).tolist()
        assert set(full) == wrote
        skipped = [i for i, p in enumerate(positions) if not 0 <= p < 100]
        assert all(bool((out[i] == 0).all()) for i in skipped)
    assert _status() == 0


# ---- attention ---------------------------------------------------------------------------------------

def _attn_case(lens, hq, hkv, D, page, dtype, kv=None, window=0, hnd=False, seed=0, qscale=1.0,
               extra_ld=0, lse=True, spare=3):
    """Runs one case and checks every output against the 64-bit statement; returns (out, lse)."""
    kv = kv or dtype
    g = _gen(seed + D + page)
    B = len(lens)
    columns = max(1, -(-max(lens) // page))
    count = B * columns + spare
    kc, vc = _cache_tensors(count, page, hkv, D, kv, g, hnd)
    table = torch.randperm(count, generator=g, device="cuda")[:B * columns].view(B, columns).int()
    bits = torch.uint8 if kv == E4M3 else torch.int16
    nan = 0x7F if kv == E4M3 else 0x7FFF
    for c in (kc, vc):  # everything that no sequence attends to is NaN
        seen = torch.zeros(count, page, dtype=torch.bool, device="cuda")
        for b, n in enumerate(lens):
            j = torch.arange(max(0, n - window) if window else 0, n, device="cuda")
            seen[table[b][j // page].long(), j % page] = True
        raw = c.view(bits)
        raw[~seen] = nan
    for b, n in enumerate(lens):  # columns outside are never read
        used = -(-n // page)
        table[b, used:] = -7
        if window and n > window:
            table[b, :(n - window) // page] = 1 << 30
    scales = [0.5 + torch.rand(hkv, device="cuda", generator=g) if kv == E4M3 else None for _ in range(2)]
    q = torch.full((B, hq * D + extra_ld), math.nan, dtype=dtype, device="cuda")
    q[:, :hq * D] = _randn((B, hq * D), dtype, g, qscale)
    out = torch.full((B, hq * D + extra_ld), 9.0, dtype=dtype, device="cuda")
    lse_t = torch.empty(B, hq, device="cuda") if lse else None
    cache = w4.kv_cache(kc, vc, *scales)
    cfg = w4.attn_config(hq, CODE[dtype], D ** -0.5, columns, window=window, ldq=hq * D + extra_ld,
                         ldo=hq * D + extra_ld)
    ws = w4.attn_workspace(cfg, cache)
    lens_t = torch.tensor(lens, dtype=torch.int32, device="cuda")
    w4.dec_attn_paged(cfg, cache, q, table, lens_t, B, out, lse_t, ws)
    assert _status() == 0
    first = (out.clone(), lse_t.clone() if lse else None)
    # the same workspace serves the next call, and equal inputs give equal bits
    out.fill_(9.0)
    w4.dec_attn_paged(cfg, cache, q, table, lens_t, B, out, lse_t, ws)
    assert _status() == 0
    assert torch.equal(first[0].view(torch.int16), out.view(torch.int16))
    if lse:
        assert torch.equal(first[1], lse_t)
    assert bool((out[:, hq * D:] == 9).all())
    G = hq // hkv
    for b, n in enumerate(lens):
        j0 = max(0, n - window) if window else 0
        for kvh in range(hkv):
            K = od.cached_tokens(kc, table[b], page, j0, n, kvh)
            V = od.cached_tokens(vc, table[b], page, j0, n, kvh)
            if kv == E4M3:
                K, V = K * scales[0][kvh].to(F64), V * scales[1][kvh].to(F64)
            for h in range(kvh * G, kvh * G + G):
                want, wlse, mag, spread = od.attn(q[b, h * D:h * D + D].to(F64), K, V, D ** -0.5)
                got = out[b, h * D:h * D + D]
                if n == 0:
                    assert bool((got == 0).all()) and (not lse or float(lse_t[b, h]) == -math.inf)
                    continue
                ds = spread * (D + 8) * 2.0 ** -23
                eps = 2 * ds + 2.0 ** -15 + (n - j0) * 2.0 ** -23 + 2.0 ** -21
                _within(got, want, want.abs() * U[dtype] + 2 * eps * mag + TINY[dtype], f"out {b},{h}")
                if lse:
                    tol = ds + (1 + abs(wlse)) * 2.0 ** -20 + (n - j0) * 2.0 ** -23
                    assert abs(float(lse_t[b, h]) - wlse) <= tol, (b, h, float(lse_t[b, h]), wlse, tol)
    return out, lse_t


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("n", [0, 1, 2, 15, 16, 17, 31, 33, 64, 100, 257])
def test_attn_lengths(n, dtype):
    _attn_case([n], 8, 2, 64, 16, dtype, seed=n)


ATTN_CASES = [
    # lens, q_heads, kv_heads, D, page, kv, window, hnd
    ([5, 0, 300, 1, 77], 8, 8, 128, 16, None, 0, False),
    ([1000, 3], 64, 8, 128, 64, None, 0, False),
    ([513, 64, 1023], 16, 1, 64, 32, None, 0, True),       # 16 rows share a head
    ([200, 90], 14, 2, 128, 16, None, 0, False),           # 7 rows
    ([130, 40], 24, 2, 64, 16, None, 0, False),            # 12 rows
    ([300, 17], 40, 1, 64, 16, None, 0, False),            # 40 rows: three row tiles
    ([100, 257], 4, 4, 80, 8, None, 0, False),             # pages end inside a tile
    ([77, 33, 5], 6, 2, 96, 5, None, 0, True),
    ([60, 61], 3, 3, 8, 1, None, 0, False),
    ([500, 2], 4, 1, 256, 16, None, 0, False),
    ([300, 450], 20, 2, 200, 24, None, 0, False),
    ([700, 0, 90], 8, 2, 128, 16, E4M3, 0, False),
    ([333], 32, 4, 64, 32, E4M3, 0, True),
    ([120, 50], 16, 1, 256, 8, E4M3, 0, False),
    ([90, 31], 6, 6, 16, 3, E4M3, 0, False),
    ([240, 10, 77], 9, 3, 112, 16, E4M3, 0, False),
    ([400, 10, 0, 129, 128], 8, 2, 64, 16, None, 128, False),
    ([1000, 37], 4, 4, 128, 16, None, 1, False),           # the newest token alone
    ([600, 333], 16, 2, 128, 16, E4M3, 100, False),
    ([50, 700], 8, 4, 72, 7, None, 33, True),
    ([900, 3, 0, 411], 24, 2, 256, 16, None, 0, False),     # two tiles of wide heads
    ([1500, 64], 32, 2, 256, 8, E4M3, 0, True),
    ([200] * 90, 18, 2, 136, 12, None, 0, False),
]


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("lens,hq,hkv,D,page,kv,window,hnd", ATTN_CASES)
def test_attn(lens, hq, hkv, D, page, kv, window, hnd, dtype):
    _attn_case(lens, hq, hkv, D, page, dtype, kv, window, hnd, seed=len(lens), extra_ld=8)


@pytest.mark.parametrize("kv", [None, E4M3], ids=str)
def test_attn_many_short_sequences(kv):
    g = torch.Generator().manual_seed(3)
    lens = torch.randint(0, 60, (700,), generator=g).tolist()
    _attn_case(lens, 2, 1, 64, 16, torch.bfloat16, kv, seed=5)


SPLITS = [
    # few items, none cut; cut by themselves; in equal shares
    ([260, 40, 300], 8), ([700], 4), ([900] * 14, 4), ([2500, 30, 2000, 1], 8),
    # more items than CTAs: whole ones (ragged, with empty sequences), and a long one among short
    (list(range(1, 300, 7)), 8), ([0, 500] * 20, 8), ([3000] + [9] * 50, 8), ([300] * 20, 8)]


@pytest.mark.parametrize("kv", [None, E4M3], ids=str)
@pytest.mark.parametrize("lens,heads", SPLITS, ids=lambda x: str(x)[:24].replace(" ", ""))
def test_attn_every_way_of_splitting(lens, heads, kv):
    """However the items are cut, the results are the statement's."""
    _attn_case(lens, heads, heads, 64 if kv else 128, 16, torch.bfloat16, kv, seed=len(lens))


def test_attn_long_sequence_is_split():
    _attn_case([70001, 19], 4, 2, 128, 64, torch.bfloat16, seed=7)


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("qscale", [0.0, 60.0])
def test_attn_flat_and_peaked_scores(qscale, dtype):
    """All scores equal, and scores that differ by hundreds (one token takes all weight)."""
    _attn_case([260, 1000], 8, 2, 64, 16, dtype, seed=9, qscale=qscale)


def test_attn_scores_that_rise_and_fall():
    """Running maxima that move at every tile, upwards in one head and downwards in the other."""
    D, n, page, dtype = 64, 4096, 16, torch.bfloat16
    ramp = torch.linspace(-40, 40, n, device="cuda")
    kc, vc = (torch.zeros(n // page, page, 2, D, dtype=dtype, device="cuda") for _ in range(2))
    kc.view(n, 2, D)[:, 0, 0], kc.view(n, 2, D)[:, 1, 0] = ramp.to(dtype), ramp.flip(0).to(dtype)
    vc.copy_(torch.randn(vc.shape, device="cuda", generator=_gen(4)))
    q = torch.zeros(1, 2 * D, dtype=dtype, device="cuda")
    q[0, 0] = q[0, D] = 8.0
    table = torch.arange(n // page, device="cuda").int()[None]
    cfg, cache = w4.attn_config(2, CODE[dtype], 1.0, n // page), w4.kv_cache(kc, vc)
    out = torch.empty_like(q)
    w4.dec_attn_paged(cfg, cache, q, table, torch.tensor([n], dtype=torch.int32, device="cuda"), 1, out,
                      None, w4.attn_workspace(cfg, cache))
    assert _status() == 0
    for h in range(2):
        want, _, mag, spread = od.attn(q[0, h * D:(h + 1) * D].to(F64), kc.view(n, 2, D)[:, h].to(F64),
                                       vc.view(n, 2, D)[:, h].to(F64), 1.0)
        eps = 2 * spread * (D + 8) * 2.0 ** -23 + 2.0 ** -15 + n * 2.0 ** -23 + 2.0 ** -21
        _within(out[0, h * D:(h + 1) * D], want, want.abs() * U[dtype] + 2 * eps * mag, f"out {h}")


def test_attn_bad_pages_and_lengths_are_reported():
    D, page, dtype = 64, 16, torch.float16
    g = _gen(2)
    kc, vc = _cache_tensors(8, page, 1, D, dtype, g)
    q = _randn((2, D), dtype, g)
    cfg, cache = w4.attn_config(1, CODE[dtype], 0.125, 3), w4.kv_cache(kc, vc)
    ws = w4.attn_workspace(cfg, cache)

    def run(table, lens):
        out = torch.empty(2, D, dtype=dtype, device="cuda")
        w4.dec_attn_paged(cfg, cache, q, torch.tensor(table, dtype=torch.int32, device="cuda"),
                          torch.tensor(lens, dtype=torch.int32, device="cuda"), 2, out, None, ws)
        return out, _status()

    good, st = run([[0, 1, 2], [3, 4, 5]], [48, 40])
    assert st == 0
    for lens in ([49, 40], [1 << 30, 40]):  # cut to the table's 48 tokens
        out, st = run([[0, 1, 2], [3, 4, 5]], lens)
        assert st == w4.W4A16_ERR_INVALID_ARG and torch.equal(out, good)
    out, st = run([[0, 1, 2], [3, 4, 5]], [-5, 40])
    assert st == w4.W4A16_ERR_INVALID_ARG and bool((out[0] == 0).all()) and torch.equal(out[1], good[1])
    for bad in (8, -1, 0x7FFFFFFF):  # a page that is not there is left out
        out, st = run([[0, bad, 2], [3, 4, 5]], [48, 40])
        assert st == w4.W4A16_ERR_INVALID_ARG and torch.equal(out[1], good[1])
        K = torch.cat([kc[0, :, 0], kc[2, :, 0]]).to(F64)
        V = torch.cat([vc[0, :, 0], vc[2, :, 0]]).to(F64)
        want, _, mag, _ = od.attn(q[0].to(F64), K, V, 0.125)
        _within(out[0], want, want.abs() * U[dtype] + mag * 2.0 ** -13 + TINY[dtype], "out")
    out, st = run([[9, 9, 9], [3, 4, 5]], [48, 40])  # no page left: an empty row
    assert st == w4.W4A16_ERR_INVALID_ARG and bool((out[0] == 0).all()) and torch.equal(out[1], good[1])


def test_attn_offsets_past_32_bits():
    """Pages beyond 2^31 elements (and 2^32 bytes) of the cache."""
    D, page, dtype = 128, 16, torch.bfloat16
    need = (1 << 31) // (page * 8 * D) + 40
    if torch.cuda.mem_get_info()[0] < 4 * need * page * 8 * D + (1 << 30):
        pytest.skip("not enough memory")
    kc, vc = (torch.empty(need, page, 8, D, dtype=dtype, device="cuda") for _ in range(2))
    g = _gen(8)
    last = torch.arange(need - 4, need, device="cuda")
    for c in (kc, vc):
        c[last] = _randn((4, page, 8, D), dtype, g)
    q = _randn((1, 8 * D), dtype, g)
    cfg, cache = w4.attn_config(8, CODE[dtype], D ** -0.5, 4), w4.kv_cache(kc, vc)
    out = torch.empty_like(q)
    w4.dec_attn_paged(cfg, cache, q, last.int()[None], torch.tensor([61], dtype=torch.int32, device="cuda"),
                      1, out, None, w4.attn_workspace(cfg, cache))
    assert _status() == 0
    for h in range(8):
        K, V = (c[last].reshape(-1, 8, D)[:61, h].to(F64) for c in (kc, vc))
        want, _, mag, _ = od.attn(q[0, h * D:(h + 1) * D].to(F64), K, V, D ** -0.5)
        _within(out[0, h * D:(h + 1) * D], want, want.abs() * U[dtype] + mag * 2.0 ** -13, f"out {h}")
    # and the append finds the same slots
    k, v = (_randn((1, 8 * D), dtype, g) for _ in range(2))
    rc = w4.rope_config(0, 8, D, CODE[dtype], None, 0)
    w4.dec_rope_append(rc, cache, None, k, v, 1, torch.zeros(1, dtype=torch.int32, device="cuda"),
                       torch.tensor([need * page - 1], device="cuda"), None)
    assert _status() == 0
    assert torch.equal(kc[need - 1, page - 1].view(-1), k[0]) and torch.equal(vc[need - 1, page - 1].view(-1), v[0])


def test_operators_on_another_stream_and_in_a_graph():
    """norm -> rope + append -> attention captured on a side stream and replayed on new inputs."""
    T, hq, hkv, D, page, dtype = 3, 8, 2, 64, 16, torch.bfloat16
    H = (hq + 2 * hkv) * D
    g = _gen(6)
    table = od.rope_table(od.rope_frequencies(D, 10000.0), 100).float().cuda()
    kc, vc = _cache_tensors(12, page, hkv, D, dtype, g)
    x, y = _randn((T, H), dtype, g), torch.empty(T, H, dtype=dtype, device="cuda")
    qo, out = (torch.empty(T, hq * D, dtype=dtype, device="cuda") for _ in range(2))
    pages = torch.arange(12, device="cuda").view(T, 4).int()
    lens = torch.tensor([5, 33, 64], dtype=torch.int32, device="cuda")
    positions, slots = lens - 1, (pages.long()[torch.arange(T), (lens - 1).long() // page] * page + (lens - 1) % page)
    cache = w4.kv_cache(kc, vc)
    rc = w4.rope_config(hq, hkv, D, CODE[dtype], table, D, ldq=H, ldk=H, ldv=H)
    ac = w4.attn_config(hq, CODE[dtype], D ** -0.5, 4)
    ws = w4.attn_workspace(ac, cache)

    def step():
        w4.dec_rms_norm(x, None, None, T, H, CODE[dtype], 1e-5, None, y)
        w4.dec_rope_append(rc, cache, y[:, :hq * D], y[:, hq * D:(hq + hkv) * D], y[:, (hq + hkv) * D:], T,
                           positions, slots, qo)
        w4.dec_attn_paged(ac, cache, qo, pages, lens, T, out, None, ws)

    step()
    torch.cuda.synchronize()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=side):
        step()
    x.copy_(_randn((T, H), dtype, g))
    want = []
    step()
    want.append(out.clone())
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want[0]) and _status() == 0
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        out.zero_()
        step()
    side.synchronize()
    assert torch.equal(out, want[0])
