"""Log probabilities, entropy and largest logits (dec_token_logprobs) against 64 bits."""
import math

import pytest
import torch

import weight_only_int4_tma_gb300 as w4
from oracle import drafts

pytestmark = pytest.mark.gpu

KINDS = {"fp16": (torch.float16, w4.DEC_LOGITS_FP16), "bf16": (torch.bfloat16, w4.DEC_LOGITS_BF16),
         "fp32": (torch.float32, w4.DEC_LOGITS_FP32)}
MARK = 7.25


def call(x, kind, factor=None, ids=None, top=0, ld=0, vocab=None, status=0, stream=None):
    """x [T, >= vocab] on the device; the five results."""
    T, V = x.shape[0], vocab or x.shape[1]
    n = ids.shape[1] if ids is not None else 0
    new = lambda *s, t=torch.float32: torch.full(s, 99, dtype=t, device="cuda")  # noqa: E731
    lp, lse, ent = new(T, max(n, 1)), new(T), new(T)
    tid, tlp = new(T, max(top, 1), t=torch.int32), new(T, max(top, 1))
    cfg = w4.logprob_config(V, KINDS[kind][1], n_ids=n, top=top, ld=ld)
    w4.dec_token_logprobs(cfg, x, factor, ids, T, lp if n else None, lse, ent, tid if top else None,
                          tlp if top else None, stream=stream)
    assert w4.w4a16_get_device_status(stream) == status
    return lp[:, :n], lse, ent, tid[:, :top], tlp[:, :top]


def close(got, want, size):
    """fp32 results: half a step of the result, and the errors of what it is made of: logits times the
    factor (2^-24 of `size`, twice), exponentials and their sums (2^-20)."""
    got, want = got.double().cpu(), torch.as_tensor(want, dtype=torch.float64)
    same = (got == want) | (torch.isnan(got) & torch.isnan(want))
    off = torch.where(same, torch.zeros_like(got), (got - want).abs())
    bound = want.abs().nan_to_num(0, 0, 0) * 2.0 ** -23 + size * 2.0 ** -22 + 2.0 ** -20
    assert bool((off <= bound).all()), (got[~(off <= bound)][:5], want[~(off <= bound)][:5])


def check(x, factor, ids, top, got, vocab=None):
    lp, lse, ent, tid, tlp = got
    for t in range(x.shape[0]):
        row = x[t, :vocab].cpu()
        f = 1.0 if factor is None else float(factor[t])
        logp, want_lse, want_ent = drafts.logprob_row(row, f)
        fin = row.double()[torch.isfinite(row)]
        size = float(fin.abs().max()) * abs(f) if len(fin) and math.isfinite(f) else 0.0
        close(lse[t], want_lse, size)
        # the entropy weighs |z - lse| by p: its terms' errors add up to a few of 2^-22 of them
        close(ent[t], want_ent, size + 30.0)
        if ids is not None:
            want = [0.0 if i < 0 else math.nan if i >= row.numel() else float(logp[i]) for i in ids[t].tolist()]
            close(lp[t], want, size)
        if top:
            order = drafts.order(row)[:top]
            assert tid[t].tolist() == order, t
            close(tlp[t], logp[order], size)


def logits(T, V, kind, seed=0, scale=3.0, ld=None):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.full((T, ld or V), math.nan, device="cuda").to(KINDS[kind][0])
    x[:, :V] = (torch.randn(T, V, generator=g, device="cuda") * scale).to(KINDS[kind][0])
    return x


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("V", [1, 2, 3, 7, 8, 9, 31, 33, 255, 257, 1000, 4097, 50001, 128000])
@pytest.mark.parametrize("T", [1, 3])
def test_lengths(kind, V, T):
    x = logits(T, V, kind, V + T)
    ids = torch.randint(0, V, (T, 2), device="cuda").int()
    top = min(V, 20)
    check(x, None, ids, top, call(x, kind, None, ids, top))


@pytest.mark.parametrize("T", [2, 9, 17, 40, 80, 153, 310, 700])
def test_row_counts(T):
    x = logits(T, 3001, "bf16", T)
    f = 0.3 + torch.rand(T, device="cuda")
    ids = torch.randint(0, 3001, (T, 1), device="cuda").int()
    check(x, f, ids, 5, call(x, "bf16", f, ids, 5))


@pytest.mark.parametrize("top", [1, 2, 3, 8, 16, 17, 31, 32])
@pytest.mark.parametrize("T,V", [(1, 32), (1, 40000), (200, 1111), (4, 600)])
def test_top(top, T, V):
    x = logits(T, V, "fp32", top + V)
    check(x, None, None, top, call(x, "fp32", None, None, top))


@pytest.mark.parametrize("kind", KINDS)
def test_alignment_and_strides(kind):
    """Rows at every offset from a 16-byte boundary, other values (NaN) between them."""
    for off in range(9):
        base = torch.full((6 * 2100 + 16,), math.nan, device="cuda").to(KINDS[kind][0])
        x = base[off: off + 5 * 2077].view(5, 2077)
        x[:, :2050] = torch.randn(5, 2050, device="cuda").to(x.dtype) * 4
        ids = torch.tensor([[0, 2049]] * 5, dtype=torch.int32, device="cuda")
        check(x, None, ids, 4, call(x, kind, None, ids, 4, ld=2077, vocab=2050), 2050)


def test_many_ids():
    x = logits(2, 500, "fp16")
    ids = torch.randint(-3, 500, (2, 3000), device="cuda").int()
    check(x, None, ids, 0, call(x, "fp16", None, ids))
    assert bool((call(x, "fp16", None, ids)[0][ids < 0] == 0).all())


def test_ids_out_of_range():
    x = logits(3, 100, "bf16")
    ids = torch.tensor([[5, 100], [-1, 7], [2 ** 31 - 1, 99]], dtype=torch.int32, device="cuda")
    check(x, None, ids, 0, call(x, "bf16", None, ids, status=w4.W4A16_ERR_INVALID_ARG))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("T", [1, 200])
def test_ties(kind, T):
    """Equal logits: the lowest index first; zeros of both signs are equal."""
    for V in (5, 700, 40000):
        x = torch.zeros((T, V), device="cuda").to(KINDS[kind][0])
        check(x, None, None, min(V, 32), call(x, kind, None, None, min(V, 32)))
        x[:, ::2] = -0.0
        check(x, None, None, min(V, 9), call(x, kind, None, None, min(V, 9)))
        x = torch.randint(0, 4, (T, V), device="cuda").to(KINDS[kind][0])
        check(x, None, None, min(V, 32), call(x, kind, None, None, min(V, 32)))


@pytest.mark.parametrize("T", [1, 160])
@pytest.mark.parametrize("order", ["ascending", "descending", "one_place"])
def test_orders_that_hide_the_largest(T, order):
    V = 60000
    x = torch.arange(V, device="cuda").float() * 1e-3
    if order == "descending":
        x = x.flip(0).contiguous()
    if order == "one_place":  # 40 large ones next to one another
        x = -x
        x[33333: 33373] = 5.0 + torch.arange(40, device="cuda") % 7
    x = x[None].repeat(T, 1)
    check(x[:1], None, None, 32, [r[:1] for r in call(x, "fp32", None, None, 32)])
    got = call(x, "fp32", None, None, 32)
    assert all(bool((r == r[:1]).all()) for r in got)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("T", [1, 160])
def test_masked_and_infinite_logits(kind, T):
    V = 5000
    rows = logits(8, V, kind, 3)
    rows[0, ::2] = -math.inf
    rows[1] = -math.inf
    rows[2] = -math.inf
    rows[2, 4321] = 1.0
    rows[3, 17] = math.inf
    rows[4, 17] = math.nan
    rows[4, 99] = math.inf
    rows[5] = torch.finfo(rows.dtype).min
    rows[6, :4990] = -math.inf
    rows[7, 5:8] = math.nan
    x = rows.repeat(-(-T // 8), 1)[:max(T, 8)].contiguous()
    ids = torch.tensor([[0, 1, 17, 4321]], dtype=torch.int32, device="cuda").repeat(x.shape[0], 1)
    if T == 1:
        for t in range(8):
            check(x[t: t + 1], None, ids[:1], 20, call(x[t: t + 1].contiguous(), kind, None, ids[:1], 20))
    else:
        check(x[:24], None, ids, 20, [r[:24] for r in call(x, kind, None, ids, 20)])


def test_factors():
    x = logits(8, 3000, "bf16", 4)
    f = torch.tensor([1.0, 0.0, -1.0, math.inf, math.nan, 1e-3, 20.0, 1e-30], device="cuda")
    ids = torch.randint(0, 3000, (8, 2), device="cuda").int()
    check(x, f, ids, 5, call(x, "bf16", f, ids, 5))


@pytest.mark.parametrize("kind", ["fp16", "bf16", "fp32"])
@pytest.mark.parametrize("top", [0, 20])
def test_odd_rows_of_many_blocks(kind, top):
    """Long rows that begin and end off 16 bytes; equal logits in all of one."""
    x = logits(5, 100003, kind, 16)
    x[3] = x[3, 7]
    x[4, 1000:] = -math.inf
    ids = torch.randint(0, 100003, (5, 3), device="cuda").int()
    check(x, None, ids, top, call(x, kind, None, ids, top))


def test_largest_factors():
    """Up to 2^127, the largest logit's neighbours included; above it NaN."""
    x = logits(3, 3000, "fp32", 14)
    f = torch.tensor([2.0 ** 127, 2.0 ** 127 * 1.5, 2.0 ** 126], device="cuda")
    ids = x.argmax(1, keepdim=True).int()
    lp, lse, ent, tid, tlp = call(x * 1e-3, "fp32", f, ids, 3)
    assert bool((lp[[0, 2]] == 0).all()) and bool((ent[[0, 2]] == 0).all()) and bool((tlp[[0, 2], 0] == 0).all())
    assert bool((lse[[0, 2]].double() == (x * 1e-3).max(1).values[[0, 2]].double() * f[[0, 2]].double()).all())
    assert all(bool(torch.isnan(r[1]).all()) for r in (lp, lse, ent, tlp))
    assert torch.equal(tid[:, 0], ids[:, 0])


@pytest.mark.parametrize("shift", [-1000.0, 1000.0, 60000.0])
def test_far_from_zero(shift):
    x = logits(3, 4000, "fp32", 5) + shift
    ids = torch.randint(0, 4000, (3, 2), device="cuda").int()
    check(x, None, ids, 3, call(x, "fp32", None, ids, 3))


def test_one_certain_token():
    """The rest's share of probability does not get lost in the sum: about 1e-5."""
    x = torch.zeros((2, 1000), device="cuda")
    x[:, 77] = 18.5
    check(x, None, torch.tensor([[77, 1]] * 2, dtype=torch.int32, device="cuda"), 2,
          call(x, "fp32", None, torch.tensor([[77, 1]] * 2, dtype=torch.int32, device="cuda"), 2))


def test_partial_outputs():
    x = logits(4, 900, "fp16", 6)
    _, lse, ent, tid, _ = call(x, "fp16", None, None, 3)
    cfg = w4.logprob_config(900, w4.DEC_LOGITS_FP16, n_ids=0, top=3)
    only = torch.full((4, 3), -1, dtype=torch.int32, device="cuda")
    w4.dec_token_logprobs(cfg, x, None, None, 4, None, None, None, only, None)
    assert torch.equal(only, tid)
    cfg = w4.logprob_config(900, w4.DEC_LOGITS_FP16, n_ids=0)
    e = torch.empty(4, device="cuda")
    w4.dec_token_logprobs(cfg, x, None, None, 4, None, None, e)
    assert torch.equal(e, ent)
    w4.dec_token_logprobs(cfg, x, None, None, 4, None, e, None)
    assert torch.equal(e, lse)
    assert w4.w4a16_get_device_status() == 0


def test_graph_and_streams():
    x = logits(30, 20000, "bf16", 7)
    ids = torch.randint(0, 20000, (30, 3), device="cuda").int()
    want = call(x, "bf16", None, ids, 10)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = call(x, "bf16", None, ids, 10, stream=s)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    cfg = w4.logprob_config(20000, w4.DEC_LOGITS_BF16, n_ids=3, top=10)
    out = [torch.zeros_like(r) for r in want]
    graph = torch.cuda.CUDAGraph()
    args = lambda: (cfg, x, None, ids, 30, out[0], out[1], out[2], out[3], out[4])  # noqa: E731
    w4.dec_token_logprobs(*args())
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        w4.dec_token_logprobs(*args())
    x.copy_(logits(30, 20000, "bf16", 8))
    graph.replay()
    check(x, None, ids, 10, out)


def test_large_offsets():
    """More than 2^31 logits in all; the last rows are right."""
    T, V = 17000, 128000
    x = torch.zeros((T, V), dtype=torch.float16, device="cuda")
    x[-2:] = logits(2, V, "fp16", 9)
    ids = torch.randint(0, V, (T, 1), device="cuda").int()
    got = call(x, "fp16", None, ids, 2)
    check(x[-2:], None, ids[-2:], 2, [r[-2:] for r in got])
    assert bool((got[1][:-2] == got[1][0]).all()) and bool((got[3][:-2] == torch.tensor([0, 1], device="cuda")).all())
