"""How exact the weights of the tree attention are: P's two 16-bit parts (csrc/tree.cuh), restated, against what
include/decode.h says of them."""
import os
import re

import numpy as np
import pytest

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "decode.h")
WEIGHTS = {"bf16": 2.0 ** -15, "fp16": 2.0 ** -19, "e4m3": 2.0 ** -20}   # of a weight, by the cache's type


def bf16(x):
    """Rounded to nearest, ties to even, and back to fp32."""
    b = x.astype(np.float32).view(np.uint32).astype(np.uint64)
    return (((b + 0x7FFF + (b >> 16 & 1)) >> 16) << 16).astype(np.uint32).view(np.float32)


def cut(x, drop):
    return (x.view(np.uint32) & np.uint32(0xFFFFFFFF << drop & 0xFFFFFFFF)).view(np.float32)


def parts(p, kind):
    one = np.float32(1)
    if kind == "bf16":
        hi = cut(p, 16)
        low = (p.astype(np.float64) * float(one + np.float32(2.0 ** -22)) - hi).astype(np.float32)   # one rounding: an fma
        return hi, bf16(low)
    c = p * (one - np.float32(2.0 ** -10)) if kind == "fp16" else p
    hi = cut(c, 13)   # fp16's subnormal numbers are cut at 2^-24
    hi = np.where(hi < 2.0 ** -14, np.floor(c.astype(np.float64) * 2.0 ** 24) * 2.0 ** -24, hi).astype(np.float32)
    low = p - cut(c, 13)
    return hi, low.astype(np.float16).astype(np.float32)


@pytest.mark.parametrize("kind", WEIGHTS)
def test_two_parts(kind):
    """Beside the parts' error there is the exponential's, 2^-22, and that of its argument's rounding, 2^-21 ln 2 where
    the argument is below 16; together they stay within the bound, or, where fp16's smallest step shows, within
    2^-30 of the row's largest weight, which is at least 2^7 there."""
    rng = np.random.default_rng(1)
    most = 2.0 ** 15 if kind != "bf16" else 2.0 ** 8
    p = np.concatenate([2.0 ** rng.uniform(-40, np.log2(most), 400000), 1 + np.arange(1 << 17) / (1 << 17)]).astype(np.float32)
    hi, low = parts(p, kind)
    off = np.abs(hi.astype(np.float64) + low - p)
    rest = 2.0 ** -22 + 2.0 ** -21 * np.log(2)
    bound = p * (WEIGHTS[kind] - rest)
    if kind != "bf16":
        bound = np.maximum(bound, 2.0 ** 7 * 2.0 ** -30)
    assert (off <= bound).all(), (np.log2(off / p).max(), p[off > bound][:5])


def test_the_header_says_so():
    with open(HEADER) as f:
        text = re.sub(r"\s*\n \*\s*", " ", f.read())
    said = re.search(r"a token's weight is exact to (2\^-\d+) of itself over a bf16 cache, (2\^-\d+) over an fp16 one and "
                     r"(2\^-\d+) over an 8-bit one", text)
    assert said and [2.0 ** int(x[2:]) for x in said.groups()] == list(WEIGHTS.values())
