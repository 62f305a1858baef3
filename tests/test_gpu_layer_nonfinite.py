"""Infinities and NaN in what the paged attention (include/decode.h) attends to, against its formula
in 64 bits: which elements are NaN or infinite follows from the formula, the others have the bits
that they have without them."""
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


class Case:
    """Sequences of `lens` tokens over a cache of pages of 16, all inputs finite."""

    def __init__(self, lens, hq, hkv, D, dtype, kv=None, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.lens, self.hq, self.hkv, self.D, self.dtype, self.page = lens, hq, hkv, D, dtype, 16
        columns = -(-max(lens) // 16)
        shape = (len(lens) * columns, 16, hkv, D)
        kv = kv or dtype
        # positive throughout: an infinity then has the same sign in every product with it
        self.k, self.v = ((0.1 + torch.rand(shape, generator=g, device="cuda")).to(kv) for _ in range(2))
        self.q = (0.1 + torch.rand((len(lens), hq * D), generator=g, device="cuda")).to(dtype)
        self.pages = torch.randperm(shape[0], generator=g, device="cuda").view(len(lens), columns).int()

    def put(self, cache, b, token, head, d, value):
        at = int(self.pages[b, token // 16]), token % 16, head, d
        cache[at] = torch.tensor(value, device="cuda").to(cache.dtype)

    def run(self):
        cache = w4.kv_cache(self.k, self.v)
        cfg = w4.attn_config(self.hq, CODE[self.dtype], self.D ** -0.5, self.pages.shape[1])
        out = torch.empty_like(self.q)
        lse = torch.empty(len(self.lens), self.hq, device="cuda")
        w4.dec_attn_paged(cfg, cache, self.q, self.pages, torch.tensor(self.lens, dtype=torch.int32, device="cuda"),
                          len(self.lens), out, lse, w4.attn_workspace(cfg, cache))
        assert w4.w4a16_get_device_status() == 0
        return out.view(-1, self.hq, self.D), lse

    def formula(self, b, h):
        """Scores and values of one row in 64 bits."""
        j = torch.arange(self.lens[b], device="cuda")
        page, slot, kvh = self.pages[b].long()[j // 16], j % 16, h // (self.hq // self.hkv)
        K, V = ((c.view(torch.uint8) if c.dtype == E4M3 else c)[page, slot, kvh].view(c.dtype).to(F64)
                for c in (self.k, self.v))
        return self.D ** -0.5 * (K * self.q.view(-1, self.hq, self.D)[b, h].to(F64)).sum(1), V


# lens, kv heads, query heads per kv head, cached type: items whole, cut by themselves, cut in equal
# shares (more items than half the CTAs), and joined in two rounds (over 32 parts)
LAYOUTS = [([5, 300], 2, 4, None), ([3000], 4, 2, None), ([1500, 4000], 50, 1, None), ([40000], 1, 12, None),
           ([300, 900], 4, 4, E4M3), ([3000], 2, 16, E4M3)]


def _case(layout, dtype, seed=0):
    lens, hkv, group, kv = layout
    return Case(lens, hkv * group, hkv, 64, dtype, kv, seed)


def _same_but(got, before, rows):
    """Rows (b, h) apart, outputs and log-sum-exps have the bits they had."""
    keep = torch.ones_like(got[1], dtype=torch.bool)
    for b, h in rows:
        keep[b, h] = False
    assert torch.equal(got[0][keep], before[0][keep]) and torch.equal(got[1][keep], before[1][keep])


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16], ids=str)
@pytest.mark.parametrize("layout", LAYOUTS, ids=str)
@pytest.mark.parametrize("where", ["first", "middle", "last"])
def test_a_nan_key_gives_nan_in_out_and_lse(layout, dtype, where):
    c = _case(layout, dtype)
    before = c.run()
    b, head = len(c.lens) - 1, c.hkv - 1
    token = {"first": 0, "middle": c.lens[b] // 2, "last": c.lens[b] - 1}[where]
    c.put(c.k, b, token, head, 7, math.nan)
    got = c.run()
    G = c.hq // c.hkv
    rows = [(b, h) for h in range(head * G, head * G + G)]
    for b, h in rows:
        assert bool(got[0][b, h].isnan().all()) and math.isnan(float(got[1][b, h])), (b, h)
    _same_but(got, before, rows)


@pytest.mark.parametrize("layout", LAYOUTS[:4], ids=str)
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16], ids=str)
def test_an_infinite_score_gives_lse_infinity(layout, dtype):
    """A key's infinity: scores of +inf where the query is positive, -inf (no weight) where negative."""
    c = _case(layout, dtype, 1)
    b, head = 0, 0
    G = c.hq // c.hkv
    if G > 1:
        c.q.view(-1, c.hq, c.D)[b, 1, 3] *= -1
    token = c.lens[b] // 3
    before = c.run()
    c.put(c.k, b, token, head, 3, math.inf)
    got = c.run()
    rows = [(b, h) for h in range(head * G, head * G + G)]
    for b, h in rows:
        s, V = c.formula(b, h)
        want = float(torch.logsumexp(s, 0))
        if want == math.inf:
            assert float(got[1][b, h]) == math.inf and bool(got[0][b, h].isnan().all())
        else:  # the token has no weight; bounds as for any row (sums of positive numbers)
            n, ds = len(s), float(s.max()) * (c.D + 8) * 2.0 ** -23
            assert abs(float(got[1][b, h]) - want) <= ds + (1 + abs(want)) * 2.0 ** -20 + n * 2.0 ** -23
            out = torch.softmax(s, 0) @ V
            eps = 2 * ds + 2.0 ** -15 + n * 2.0 ** -23 + 2.0 ** -21
            assert bool(((got[0][b, h].to(F64) - out).abs() <= out * (U[dtype] + 2 * eps) + 2.0 ** -25).all())
    assert G == 1 or float(got[1][b, 1]) < math.inf
    _same_but(got, before, rows)


@pytest.mark.parametrize("kv", [None, E4M3], ids=str)
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16], ids=str)
@pytest.mark.parametrize("value,lse", [(math.inf, math.inf), (-math.inf, -math.inf), (math.nan, math.nan)])
def test_an_infinite_query_reaches_every_score(value, lse, dtype, kv):
    """All scores +inf: out NaN, lse +inf.  All -inf: no weight anywhere, out 0, lse -inf.  Large
    finite values of the other sign beside the infinity change nothing."""
    c = Case([777], 4, 2, 64, dtype, kv, 2)
    before = c.run()
    row = c.q.view(-1, c.hq, c.D)[0, 1]
    row[:] = math.copysign(torch.finfo(dtype).max / 16, -value)
    row[:60] = 0.5
    row[9] = value
    got = c.run()
    assert torch.equal(got[1][0, 1].cpu(), torch.tensor(lse)) or (math.isnan(lse) and bool(got[1][0, 1].isnan()))
    if value == -math.inf:
        assert bool((got[0][0, 1] == 0).all())
    else:
        assert bool(got[0][0, 1].isnan().all())
    _same_but(got, before, [(0, 1)])


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16], ids=str)
@pytest.mark.parametrize("layout", LAYOUTS[:4], ids=str)
@pytest.mark.parametrize("scores", ["flat", "spread", "below"])
def test_an_infinite_value_gives_its_infinity(layout, dtype, scores):
    """Values +inf, -inf, both and NaN in columns of their own; the other columns keep their bits.
    flat: all weights are 1; below: the tokens with these values weigh some 2^-27 of the largest."""
    c = _case(layout, dtype, 3)
    b, head = len(c.lens) - 1, 0
    n, G = c.lens[b], c.hq // c.hkv
    at = [0, n // 3, n // 2, n - 1]
    if scores == "flat":
        c.q.zero_()
    if scores == "below":  # one key apart is larger: e^18.5 is 2^26.7
        c.k.fill_(0.25)
        c.q.fill_(0.5)
        c.put(c.k, b, n // 4, head, slice(0, 64), 0.25 + 18.5 / 4)
    before = c.run()
    for j, (d, value) in enumerate([(5, math.inf), (17, -math.inf), (40, math.inf), (63, math.nan)]):
        c.put(c.v, b, at[j], head, d, value)
    c.put(c.v, b, at[3], head, 40, -math.inf)
    out, lse = c.run()
    assert torch.equal(lse, before[1])
    for h in range(head * G, head * G + G):
        s, V = c.formula(b, h)
        want = torch.softmax(s, 0) @ V
        row = out[b, h].to(F64)
        odd = ~want.isfinite()
        assert odd.nonzero().squeeze(1).tolist() == [5, 17, 40, 63]
        assert torch.equal(row[[5, 17]], want[[5, 17]]) and bool(row[[40, 63]].isnan().all()), row[odd]
        assert torch.equal(out[b, h][~odd], before[0][b, h][~odd])
    _same_but((out, lse), before, [(b, h) for h in range(head * G, head * G + G)])


def test_an_infinite_value_before_the_maximum_moves():
    """The sums so far are scaled when a larger score arrives: an infinity among them stays one."""
    for dtype in (torch.float16, torch.bfloat16):
        c = Case([2000], 1, 1, 64, dtype, seed=4)
        ramp = torch.linspace(0.0, 4.0, 2000, device="cuda")  # scores rise by 16
        c.q.fill_(0.5)
        j = torch.arange(2000, device="cuda")
        c.k[c.pages[0].long()[j // 16], j % 16, 0] = ramp[:, None].to(dtype)
        c.put(c.v, 0, 3, 0, 8, -math.inf)
        out, _ = c.run()
        assert float(out[0, 0, 8]) == -math.inf and int((~out.isfinite()).sum()) == 1
