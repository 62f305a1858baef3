"""Limits of the decoder-layer operators that only the host checks (include/decode.h)."""
import pytest

import weight_only_int4_tma_gb300 as w4
from weight_only_int4_tma_gb300 import build as w4build

F = 1 << 20  # an aligned address that is never dereferenced


@pytest.mark.parametrize("B,want", [(1 << 27, w4.W4A16_ERR_UNSUPPORTED), (0x7FFFFFFF, w4.W4A16_ERR_UNSUPPORTED)])
def test_attention_refuses_2_27_sequences(B, want):
    w4build.build()
    cache = w4.KvCache(F, F, None, None, 64 * 256, 256, 64, 64 * 256, 256, 64, 10, 64, 4, 64, 0, 0)
    cfg = w4.AttnConfig(8, 0, 20, 0, 0.125, 0, 0, 0, 0)
    assert w4.lib().dec_attn_paged(cfg, cache, F, F, F, B, F, None, F, 1 << 40, None) == want
