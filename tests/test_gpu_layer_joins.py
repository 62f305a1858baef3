"""The paged attention's partial results (include/decode.h): values that tell where in a sequence they come
from, so that a part lost, doubled or joined with the wrong weight shows.

The value of a token is 1 in one channel and 0 in the others, channel after channel along the sequence:
an output is the share of the weights that its stretch of tokens has.  All terms are positive, and
errors relative: U for the stored type, 2 ds for the scores (ds = (D + 8) 2^-23 of the largest sum
|q k|, in numerator and denominator), 2^-15 for the weights' two parts, and 2^-23 for each addition
on the way of a term: a warp adds two products of at most 2^8 tokens of a part, then 8 warps and two
rounds of at most 32 parts are joined: under 2^10.  With equal scores all of that is exact but the
joins' factors (2^-21) and the quotient."""
import math

import pytest
import torch

import weight_only_int4_tma_gb300 as w4

pytestmark = pytest.mark.gpu

F64 = torch.float64
E4M3 = torch.float8_e4m3fn
U = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
CODE = {torch.float16: w4.W4A16_FP16, torch.bfloat16: w4.W4A16_BF16}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from weight_only_int4_tma_gb300 import build
    build.build()


# one item of over 32 parts by itself, several of them, and in the line of equal shares among
# items that are cut too (more items than half the CTAs), where its first and last CTA hold others
LONG = [([70001], 1, 1), ([40000, 50001], 2, 4), ([500] * 45 + [70001] + [500] * 45, 1, 2),
        ([70001] + [300] * 100, 1, 1), ([900] * 30 + [60001, 1] + [900] * 30 + [0, 50000], 2, 12)]


def _inputs(lens, hkv, group, D, dtype, kv, flat, page=16):
    g = torch.Generator(device="cuda").manual_seed(len(lens) + D)
    columns = [-(-n // page) for n in lens]
    count = sum(columns)
    perm = torch.randperm(count, generator=g, device="cuda").int()
    pages = torch.full((len(lens), max(columns)), -1, dtype=torch.int32, device="cuda")
    k = torch.randn((count, page, hkv, D), generator=g, device="cuda").to(dtype).to(kv)
    v = torch.zeros((count, page, hkv, D), device="cuda")
    at, channels = 0, []
    for b, n in enumerate(lens):
        pages[b, :columns[b]] = perm[at:at + columns[b]]
        at += columns[b]
        j = torch.arange(n, device="cuda")
        channels.append(j * D // max(n, 1))
        v[pages[b].long()[j // page], j % page, :, channels[b]] = 1
    q = torch.zeros((len(lens), hkv * group * D), dtype=dtype, device="cuda")
    if not flat:
        q = torch.randn(q.shape, generator=g, device="cuda").to(dtype)
    return q, k, v.to(kv), pages, channels


@pytest.mark.parametrize("flat", [True, False], ids=["flat", "spread"])
@pytest.mark.parametrize("dtype,kv,D", [(torch.bfloat16, None, 128), (torch.float16, None, 64),
                                        (torch.bfloat16, E4M3, 64), (torch.float16, E4M3, 128),
                                        (torch.bfloat16, None, 256)], ids=str)
@pytest.mark.parametrize("lens,hkv,group", LONG, ids=lambda x: str(x)[:20].replace(" ", ""))
def test_every_part_counts(lens, hkv, group, dtype, kv, D, flat):
    hq, page = hkv * group, 16
    q, k, v, pages, channels = _inputs(lens, hkv, group, D, dtype, kv or dtype, flat)
    cache, cfg = w4.kv_cache(k, v), w4.attn_config(hq, CODE[dtype], D ** -0.5, pages.shape[1])
    out, lse = torch.empty_like(q), torch.empty(len(lens), hq, device="cuda")
    w4.dec_attn_paged(cfg, cache, q, pages, torch.tensor(lens, dtype=torch.int32, device="cuda"), len(lens), out, lse,
                      w4.attn_workspace(cfg, cache))
    assert w4.w4a16_get_device_status() == 0
    out = out.view(len(lens), hq, D)
    for b, n in enumerate(lens):
        if n == 0:
            assert bool((out[b] == 0).all()) and bool((lse[b] == -math.inf).all())
            continue
        j = torch.arange(n, device="cuda")
        for h in range(0, hq, max(1, hq // 3)):
            K = k.view(torch.uint8 if kv else k.dtype)[pages[b].long()[j // page], j % page, h // group].view(k.dtype).to(F64)
            row = q[b, h * D:(h + 1) * D].to(F64)
            s = (K @ row) * D ** -0.5
            p = torch.softmax(s, 0)
            want = torch.zeros(D, dtype=F64, device="cuda").index_add_(0, channels[b], p)
            ds = float((K.abs() @ row.abs()).max()) * D ** -0.5 * (D + 8) * 2.0 ** -23
            eps = 2.0 ** -20 if flat else 2 * ds + 2.0 ** -15 + 2.0 ** -13 + 2.0 ** -21
            tol = want * (U[dtype] + eps) + 2.0 ** -25
            off = (out[b, h].to(F64) - want).abs()
            assert bool((off <= tol).all()), (b, h, float((off / tol).max()))
            ltol = ds + (1 + math.log(n)) * 2.0 ** -20 + (0 if flat else 2.0 ** -13)
            assert abs(float(lse[b, h]) - float(torch.logsumexp(s, 0))) <= ltol
            if n >= 40000:  # the statement without any 500 of the tokens is another one
                for first in range(0, n - 500, n // 7):
                    left = p.clone()
                    left[first:first + 500] = 0
                    less = torch.zeros_like(want).index_add_(0, channels[b], left)
                    assert bool(((less - want).abs() > 4 * tol).any())
