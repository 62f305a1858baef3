"""Forms of the decoder-layer operators' calls (include/decode.h) that a server meets besides the plain
ones: strided rows and no weight for the 8-bit norms, four pieces per thread with the last ones
empty, wide block tables, keys and values laid out apart, two streams, graphs whose lengths move from one
way of splitting to another, and two tokens for one slot.

Tolerances: the norm's sums take at most 2^8 roundings of 2^-24, halved by the root, and a few for the
products: NORM = 2^-16 relative; U, half a step of the stored type."""
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
NORM = 2.0 ** -16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from weight_only_int4_tma_gb300 import build
    build.build()


def _randn(shape, dtype, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


# pieces of 8 values: 513 and 1025 (one thread has the last), 528 (a part of a warp), 2049 and 3500
# (four per thread of rows beyond 2048 pieces, few and many rows)
NORM_SHAPES = [(1300, 4104), (1300, 8192), (1250, 8200), (1300, 4224), (3, 16416), (2, 28000), (400, 16416)]


def _norm_case(M, H, dtype, ldx, ldr, weight):
    x, r = _randn((M, ldx or H), dtype, M), _randn((M, ldr or H), dtype, H, 3.0)
    w = 1 + _randn(H, dtype, 1, 0.2) if weight else None
    rout = torch.full_like(r, 7.0)
    h, y = od.rms_norm(x[:, :H], r[:, :H], w, 1e-5)
    return x, r, w, rout, h, y


def _check_rout(rout, h, H, dtype):
    off = (rout[:, :H].to(F64) - h).abs()
    assert bool((off <= h.abs() * (U[dtype] + 2.0 ** -23) + 2.0 ** -25).all())
    assert bool((rout[:, H:] == 7).all())


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("M,H", NORM_SHAPES)
def test_norm_of_long_rows(M, H, dtype):
    x, r, w, rout, h, want = _norm_case(M, H, dtype, 0, 0, True)
    y = torch.empty_like(x)
    w4.dec_rms_norm(x, r, w, M, H, CODE[dtype], 1e-5, rout, y)
    assert w4.w4a16_get_device_status() == 0
    assert bool(((y.to(F64) - want).abs() <= want.abs() * (U[dtype] + NORM) + 2.0 ** -25).all())
    _check_rout(rout, h, H, dtype)


STRIDED = [(M, H, 0, 0, True) for M, H in NORM_SHAPES] + [
    (9, 64, 72, 80, True), (9, 1152, 1160, 1152, False), (300, 512, 1024, 520, False), (1300, 4224, 4232, 4240, True),
    (1, 8192, 0, 0, False)]


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("M,H,ldx,ldr,weight", STRIDED)
def test_norm_i8_strides_and_no_weight(M, H, ldx, ldr, weight, dtype):
    x, r, w, rout, h, y = _norm_case(M, H, dtype, ldx, ldr, weight)
    codes, s = torch.empty(M, H, dtype=torch.int8, device="cuda"), torch.empty(M, device="cuda")
    w4.dec_rms_norm_i8(x, r, w, M, H, CODE[dtype], 1e-5, rout, codes, s, ldx=ldx, ldr=ldr)
    assert w4.w4a16_get_device_status() == 0
    _, scale = od.quantize_i8(y)
    assert bool(((s.to(F64) - scale).abs() <= scale * 2 * NORM).all())
    assert bool(((codes.to(F64) - y / scale[:, None]).abs() <= 0.5 + 127 * 4 * NORM).all())
    _check_rout(rout, h, H, dtype)


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("M,H,ldx,ldr,weight", [c for c in STRIDED if c[1] % 32 == 0])
def test_norm_mx_strides_and_no_weight(M, H, ldx, ldr, weight, dtype):
    x, r, w, rout, h, y = _norm_case(M, H, dtype, ldx, ldr, weight)
    codes = torch.empty(M, H, dtype=torch.uint8, device="cuda")
    s = torch.empty(M, H // 32, dtype=torch.uint8, device="cuda")
    w4.dec_rms_norm_mx(x, r, w, M, H, CODE[dtype], 1e-5, rout, codes, s, ldx=ldx, ldr=ldr)
    assert w4.w4a16_get_device_status() == 0
    lo, hi = od.quantize_mx(y * (1 - 2 * NORM))[1], od.quantize_mx(y * (1 + 2 * NORM))[1]
    e = s.to(F64) - 127
    assert bool(((e == lo) | (e == hi)).all())
    z = (y.view(M, -1, 32) * torch.exp2(-e)[:, :, None]).view(M, H).clamp(-448, 448)
    half = torch.exp2(torch.floor(torch.log2(z.abs().clamp(min=2.0 ** -6))) - 4)  # of E4M3's step
    assert bool(((codes.view(E4M3).to(F64) - z).abs() <= half + z.abs() * 2 * NORM).all())
    _check_rout(rout, h, H, dtype)


def _close(out, q, K, V, dtype):
    """One row of attention against the statement: a score is a sum of D products, weights are carried
    to 2^-15, one addition of 2^-23 per token, exp and the joins 2^-21."""
    want, _, mag, spread = od.attn(q.to(F64), K.to(F64), V.to(F64), len(q) ** -0.5)
    eps = 2 * spread * (len(q) + 8) * 2.0 ** -23 + 2.0 ** -15 + len(K) * 2.0 ** -23 + 2.0 ** -21
    assert bool(((out.to(F64) - want).abs() <= want.abs() * U[dtype] + 2 * eps * mag + 2.0 ** -25).all())


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
def test_keys_and_values_laid_out_apart_and_a_wide_table(dtype):
    """Keys [page][slot][head], values [page][head][slot] with gaps, a block table of wider rows."""
    B, hq, hkv, D, page, lens = 3, 8, 2, 64, 16, [100, 3, 77]
    columns, n = 7, 30
    k = _randn((n, page, hkv, D), dtype, 1)
    wide = _randn((n, hkv + 1, page + 2, D + 8), dtype, 2)
    v = wide[:, :hkv, :page, :D].transpose(1, 2)
    before = wide.clone()
    table = torch.full((B, columns + 5), -9, dtype=torch.int32, device="cuda")
    table[:, :columns] = torch.randperm(n, device="cuda")[:B * columns].view(B, columns)
    lens_t = torch.tensor(lens, dtype=torch.int32, device="cuda")
    cache = w4.kv_cache(k, v)
    pos = (lens_t - 1).long()
    slots = table.gather(1, (pos // page)[:, None]).squeeze(1).long() * page + pos % page
    new = [_randn((B, hkv * D), dtype, s) for s in (3, 4)]
    w4.dec_rope_append(w4.rope_config(0, hkv, D, CODE[dtype], None, 0), cache, None, *new, B,
                       torch.zeros(B, dtype=torch.int32, device="cuda"), slots, None)
    assert torch.equal(k[slots // page, slots % page].view(B, -1), new[0])
    assert torch.equal(v[slots // page, slots % page].reshape(B, -1), new[1])
    gaps = torch.ones_like(wide, dtype=torch.bool)
    gaps[:, :hkv, :page, :D] = False
    assert torch.equal(wide[gaps], before[gaps])
    q, out = _randn((B, hq * D), dtype, 5), torch.empty(B, hq * D, dtype=dtype, device="cuda")
    cfg = w4.attn_config(hq, CODE[dtype], D ** -0.5, columns, ld_table=columns + 5)
    w4.dec_attn_paged(cfg, cache, q, table, lens_t, B, out, None, w4.attn_workspace(cfg, cache))
    assert w4.w4a16_get_device_status() == 0
    for b in range(B):
        for h in range(hq):
            K, V = (od.cached_tokens(c, table[b], page, 0, lens[b], h // 4) for c in (k, v))
            _close(out[b, h * D:(h + 1) * D], q[b, h * D:(h + 1) * D], K, V, dtype)


def _attention(B, hq, hkv, D, columns, dtype, seed):
    page = 16
    k, v = (_randn((B * columns, page, hkv, D), dtype, seed + s) for s in range(2))
    table = torch.randperm(B * columns, device="cuda").view(B, columns).int()
    q, out = _randn((B, hq * D), dtype, seed + 2), torch.empty(B, hq * D, dtype=dtype, device="cuda")
    cache, cfg = w4.kv_cache(k, v), w4.attn_config(hq, CODE[dtype], D ** -0.5, columns)
    return k, v, table, q, out, cache, cfg, w4.attn_workspace(cfg, cache)


def test_two_streams_with_a_workspace_each():
    """Calls that may overlap, split in parts both: each result is that of the call alone."""
    dtype, sides = torch.bfloat16, []
    for i, (B, n) in enumerate(((2, 9000), (5, 3000))):
        k, v, table, q, out, cache, cfg, ws = _attention(B, 16, 2, 128, -(-n // 16), dtype, 10 * i)
        lens = torch.full((B,), n, dtype=torch.int32, device="cuda")
        call = lambda o, w, a=(cfg, cache, q, table, lens, B): w4.dec_attn_paged(*a, o, None, w)  # noqa: E731
        alone = torch.empty_like(out)
        call(alone, ws)
        sides.append((torch.cuda.Stream(), call, out, ws, alone, (k, v)))
    torch.cuda.synchronize()
    for _ in range(20):
        for stream, call, out, ws, _, _ in sides:
            with torch.cuda.stream(stream):
                out.zero_()
                call(out, ws)
        torch.cuda.synchronize()
        for _, _, out, _, alone, _ in sides:
            assert torch.equal(out, alone)
    assert w4.w4a16_get_device_status() == 0


def test_a_graph_whose_lengths_move_between_the_splits():
    """One captured call, replayed for lengths whose items are whole, cut by themselves, cut in equal
    shares, joined in two rounds, and empty: the bits of a call by itself."""
    dtype, B, columns = torch.float16, 12, 1300
    k, v, table, q, out, cache, cfg, ws = _attention(B, 24, 8, 64, columns, dtype, 3)
    lens = torch.ones(B, dtype=torch.int32, device="cuda")
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    call = lambda o, w: w4.dec_attn_paged(cfg, cache, q, table, lens, B, o, None, w)  # noqa: E731
    call(out, ws)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        call(out, ws)
    for now in ([1] * 12, [4000] * 12, [20800] + [3] * 11, [300] * 12, [0] * 12, [20000] * 6 + [0] * 6, [20800] + [0] * 11,
                list(range(100, 1300, 100)), [0, 17] * 6):
        lens.copy_(torch.tensor(now, dtype=torch.int32))
        want = torch.empty_like(out)
        call(want, w4.attn_workspace(cfg, cache))
        for _ in range(2):
            out.fill_(9.0)
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, want), now
        b = max(range(B), key=lambda i: now[i])
        for h in (0, 23):
            K, V = (od.cached_tokens(c, table[b], 16, 0, now[b], h // 3) for c in (k, v))
            _close(out[b, h * 64:(h + 1) * 64], q[b, h * 64:(h + 1) * 64], K, V, dtype)
    assert w4.w4a16_get_device_status() == 0


@pytest.mark.parametrize("D,rot", [(128, 128), (80, 40)])  # both kernels
def test_tokens_that_share_a_slot_leave_values_of_them_alone(D, rot):
    """Which of two tokens' values a shared slot keeps may differ from value to value, and is one of
    theirs for each; every other slot is as without them."""
    T, h, page, dtype = 600, 4, 16, torch.bfloat16
    table = od.rope_table(od.rope_frequencies(rot, 10000.0), 700).float().cuda()
    k, v = (_randn((T, h * D), dtype, s) for s in range(2))
    kc, vc = (torch.zeros(T // page + 1, page, h, D, dtype=dtype, device="cuda") for _ in range(2))
    ko = torch.empty_like(k)
    slots = torch.arange(T, device="cuda")
    slots[1::2] = slots[0::2]  # pairs of tokens
    w4.dec_rope_append(w4.rope_config(0, h, D, CODE[dtype], table, rot), w4.kv_cache(kc, vc), None, k, v, T,
                       torch.arange(T, device="cuda").int(), slots, None, ko)
    assert w4.w4a16_get_device_status() == 0
    for c, new in ((kc, ko), (vc, v)):
        got = c.view(-1, h * D)
        assert bool(((got[0:T:2] == new[0::2]) | (got[0:T:2] == new[1::2])).all())
        assert bool((got[1:T:2] == 0).all()) and bool((got[T:] == 0).all())
