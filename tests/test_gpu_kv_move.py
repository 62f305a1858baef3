"""Moves of cached tokens (dec_kv_move) against one move after another."""
import random

import pytest
import torch

import weight_only_int4_tma_gb300 as w4
from oracle import drafts

pytestmark = pytest.mark.gpu

DT = {"fp16": torch.float16, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}


def raw(x):
    return x.view(torch.uint8 if x.dtype == torch.float8_e4m3fn else torch.int16)


def cache(pages, page, heads, d, kv, seed=0, heads_first=False):
    """Random bits, NaN patterns among them: a move copies bits."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    shape = (pages, heads, page, d) if heads_first else (pages, page, heads, d)
    es = 1 if kv == "e4m3" else 2
    out = []
    for _ in range(2):
        b = torch.randint(0, 256, (*shape[:-1], shape[-1] * es), generator=g, device="cuda", dtype=torch.uint8)
        x = b.view(DT[kv])
        out.append(x.transpose(1, 2) if heads_first else x)
    return out


def i64(v):
    return torch.tensor(v, dtype=torch.int64, device="cuda")


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def run(k, v, src, dst, starts, status=0, stream=None):
    page = k.shape[1]
    want = [drafts.move(raw(x), src, dst, starts, page) for x in (k, v)]
    w4.dec_kv_move(w4.kv_cache(k, v), i64(src), i64(dst), i32(starts), len(starts) - 1, len(src), stream=stream)
    assert w4.w4a16_get_device_status(stream) == status
    assert torch.equal(raw(k), want[0]) and torch.equal(raw(v), want[1])


@pytest.mark.parametrize("kv", DT)
@pytest.mark.parametrize("heads,d", [(1, 16), (8, 128), (3, 80), (2, 256), (32, 64)])
@pytest.mark.parametrize("page", [1, 5, 16, 64])
def test_accepted_paths(kv, heads, d, page):
    rng = random.Random(heads * d + page)
    per = -(-96 // page)
    src, dst, starts = [], [], [0]
    for b in range(7):
        first, ctx = b * per * page, rng.randrange(20)
        path = sorted(rng.sample(range(64), rng.choice([0, 1, 3, 8, 20, 64])))
        src += [first + ctx + i for i in path]
        dst += [first + ctx + j for j in range(len(path))]
        starts.append(len(src))
    run(*cache(7 * per, page, heads, d, kv, page, heads_first=page == 16), src, dst, starts)


def test_order_of_moves():
    """Sources that an earlier move wrote, one destination twice, a rotation through a spare slot."""
    src = [3, 5, 7, 9, 9, 1, 2, 20, 21, 22, 23, 24, 25, 26, 27, 28, 29]
    dst = [5, 7, 9, 11, 3, 3, 3, 21, 22, 23, 24, 25, 26, 27, 28, 29, 20]
    run(*cache(4, 8, 2, 64, "bf16"), src, dst, [0, 7, 17])
    rng = random.Random(5)
    src, dst = ([rng.randrange(32) for _ in range(200)] for _ in range(2))
    run(*cache(2, 16, 2, 64, "fp16"), src, dst, [0, 200])


def test_nothing_to_move():
    run(*cache(4, 8, 2, 64, "bf16"), [-1, 4, -1], [3, -1, -1], [0, 3])
    run(*cache(4, 8, 2, 64, "bf16"), [4, 5, 6], [1, 2, 3], [1, 1, 2, 2])       # moves 0 and 2 are in no group
    k, v = cache(4, 8, 2, 64, "bf16")
    w4.dec_kv_move(w4.kv_cache(k, v), i64([1]), i64([2]), i32([0]), 0, 1)
    w4.dec_kv_move(w4.kv_cache(k, v), i64([1]), i64([2]), i32([0, 0]), 1, 0)
    assert w4.w4a16_get_device_status() == 0


def test_out_of_range():
    bad = w4.W4A16_ERR_INVALID_ARG
    run(*cache(4, 8, 2, 64, "bf16"), [1, 32, 3], [2, 4, 1 << 40], [0, 3], bad)
    # groups that are descending, negative or too long move nothing; the others do
    for starts in ([0, 1, 5, 3], [-1, 1, 2, 3], [0, 2, 1, 3]):
        k, v = cache(4, 8, 2, 64, "bf16")
        want = [raw(x).clone() for x in (k, v)]
        src, dst = [1, 2, 3], [11, 12, 13]
        for a, b in zip(starts[:-1], starts[1:]):
            if 0 <= a <= b <= 3:
                for x in want:
                    for i in range(a, b):
                        x[1, dst[i] - 8] = x[0, src[i]]
        w4.dec_kv_move(w4.kv_cache(k, v), i64(src), i64(dst), i32(starts), 3, 3)
        assert w4.w4a16_get_device_status() == bad
        assert torch.equal(raw(k), want[0]) and torch.equal(raw(v), want[1])


def test_many_groups():
    B = 70000
    k, v = cache(2 * B, 1, 1, 16, "bf16")
    src, dst = torch.arange(B) * 2, torch.arange(B) * 2 + 1
    w4.dec_kv_move(w4.kv_cache(k, v), src.cuda(), dst.cuda(), torch.arange(B + 1).int().cuda(), B, B)
    assert w4.w4a16_get_device_status() == 0
    for x in (k, v):
        assert torch.equal(raw(x)[0::2], raw(x)[1::2])


def test_offsets_past_32_bits():
    stride = (1 << 32) + 512
    buf = torch.zeros(2 * stride + 16 * 64, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    x = buf.as_strided((3, 16, 1, 64), (stride, 64, 64, 1))
    raw(x).random_(0, 255)
    want = raw(x)[2, 5].clone(), raw(x)[0, 1].clone()
    w4.dec_kv_move(w4.kv_cache(x, x), i64([37, 1]), i64([3, 20]), i32([0, 2]), 1, 2)
    assert w4.w4a16_get_device_status() == 0
    assert torch.equal(raw(x)[0, 3], want[0]) and torch.equal(raw(x)[1, 4], want[1])


def test_stream_and_graph():
    s = torch.cuda.Stream()
    k, v = cache(4, 8, 2, 64, "bf16")
    torch.cuda.synchronize()
    run(k, v, [9, 12], [8, 9], [0, 2], stream=s)
    c, src, dst, starts = w4.kv_cache(k, v), i64([17, 18]), i64([3, 4]), i32([0, 2])
    want = [drafts.move(raw(x), [20, 25], [5, 6], [0, 2], 8) for x in (k, v)]
    w4.dec_kv_move(c, src, src, starts, 1, 2)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        w4.dec_kv_move(c, src, dst, starts, 1, 2)
    src.copy_(i64([20, 25]))
    dst.copy_(i64([5, 6]))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(raw(k), want[0]) and torch.equal(raw(v), want[1])
