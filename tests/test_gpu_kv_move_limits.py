"""Moves of cached tokens (dec_kv_move) at the ends of its ranges: the last move numbers, far pages."""
import pytest
import torch

import weight_only_int4_tma_gb300 as w4
from oracle import drafts

from test_gpu_kv_move import cache, i32, i64, raw

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("count", [1, 5, 7, 8, 9, 20])
def test_last_move_numbers(count):
    """A group that ends with move 2^31 - 2, the last that there can be."""
    N = 2 ** 31 - 1
    k, v = cache(4, 8, 2, 64, "bf16")
    src, dst = (torch.full((N,), -1, dtype=torch.int64, device="cuda") for _ in range(2))
    a, b = [(3 * i) % 31 for i in range(count)], [(7 * i + 1) % 31 for i in range(count)]
    src[N - count:], dst[N - count:] = i64(a), i64(b)
    want = [drafts.move(raw(x), a, b, [0, count], 8) for x in (k, v)]
    w4.dec_kv_move(w4.kv_cache(k, v), src, dst, i32([N - count, N]), 1, N)
    assert w4.w4a16_get_device_status() == 0
    assert torch.equal(raw(k), want[0]) and torch.equal(raw(v), want[1])


def test_far_pages_of_keys_and_values():
    """Keys and values apart, each with pages more than 2^32 bytes from one another."""
    stride = (1 << 32) + 512
    k, v = (torch.zeros(2 * stride + 16 * 64, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
            .as_strided((3, 16, 1, 64), (stride, 64, 64, 1)) for _ in range(2))
    for x in (k, v):
        raw(x).random_(0, 255)
    src, dst = [37, 1, 20, 33], [3, 20, 36, 47]
    want = [drafts.move(raw(x).contiguous(), src, dst, [0, 2], 16) for x in (k, v)]
    want = [drafts.move(x, src, dst, [2, 4], 16) for x in want]
    w4.dec_kv_move(w4.kv_cache(k, v), i64(src), i64(dst), i32([0, 2]), 1, 4)
    w4.dec_kv_move(w4.kv_cache(k, v), i64(src), i64(dst), i32([2, 4]), 1, 4)
    assert w4.w4a16_get_device_status() == 0
    assert torch.equal(raw(k), want[0]) and torch.equal(raw(v), want[1])
