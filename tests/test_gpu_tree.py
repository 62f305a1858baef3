"""Attention of drafted tokens (dec_attn_tree) against its definition in 64 bits."""
import math
import random

import pytest
import torch

import weight_only_int4_tma_gb300 as w4
from oracle import drafts

pytestmark = pytest.mark.gpu

T16 = {"fp16": torch.float16, "bf16": torch.bfloat16}
KV = dict(T16, e4m3=torch.float8_e4m3fn)
CODE = {"fp16": w4.W4A16_FP16, "bf16": w4.W4A16_BF16}
MARK = 7.25  # what stands in rows that must be left as they were


def tree_words(n, rng, wide=6):
    """A random tree's mask words, every token's parent one of the `wide` before it."""
    return w4.tree_mask([i - 1 - rng.randrange(min(i + 1, wide)) if i else -1 for i in range(n)])


class Case:
    """A batch: (context, drafted) per sequence, random pages, everything that no row sees NaN."""

    def __init__(self, seqs, hq, hkv, d, dtype="bf16", kv=None, page=16, window=0, sinks=0, mask="tree",
                 pad=(0, 0), seed=0, heads_first=False, ldq=0, ldo=0, scale=None, spread=1.5):
        rng, g = random.Random(seed), torch.Generator(device="cuda").manual_seed(seed)
        self.seqs, self.hq, self.hkv, self.d, self.page = seqs, hq, hkv, d, page
        self.window, self.sinks, self.dtype, self.kv = window, sinks, dtype, kv or dtype
        self.scale = d ** -0.5 if scale is None else scale
        starts = [pad[0]]
        for _, n in seqs:
            starts.append(starts[-1] + n)
        self.T, self.starts = starts[-1] + pad[1], starts
        self.words = None
        if mask is not None:
            self.words = [[w % (1 << 64) for w in (tree_words(n, rng) if mask == "tree" else mask(n, rng))] for _, n in seqs]
        columns = max(1, max(-(-(c + n) // page) for c, n in seqs)) + 1
        count = len(seqs) * columns + 3
        randn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        self.q = torch.full((self.T, max(ldq, hq * d)), MARK, device="cuda").to(T16[dtype])
        self.q[:, : hq * d] = (randn(self.T, hq * d) * spread).to(T16[dtype])
        order = list(range(count))
        rng.shuffle(order)
        self.pages = torch.tensor(order[: len(seqs) * columns], dtype=torch.int32).view(len(seqs), columns)
        shape = (count, hkv, page, d) if heads_first else (count, page, hkv, d)
        self.k, self.v = (torch.full(shape, math.nan, device="cuda").to(KV[self.kv]) for _ in range(2))
        if heads_first:
            self.k, self.v = self.k.transpose(1, 2), self.v.transpose(1, 2)
        for b, (c, n) in enumerate(seqs):  # only the tokens of the sequences hold numbers
            if n == 0:
                continue
            j = torch.arange(c + n)
            at = (self.pages[b][j // page].long().cuda(), (j % page).cuda())
            for x in (self.k, self.v):
                new = (randn(c + n, hkv, d) * (16.0 if self.kv == "e4m3" else 1.0)).to(KV[self.kv])
                bits(x)[at] = bits(new)
        self.ks = self.vs = None
        if self.kv == "e4m3":
            self.ks, self.vs = (0.04 + 0.03 * torch.rand(hkv, generator=g, device="cuda") for _ in range(2))
        self.lens = torch.tensor([c + n if n else -5 for c, n in seqs], dtype=torch.int32, device="cuda")
        self.out = torch.full((self.T, max(ldo, hq * d)), MARK, device="cuda").to(T16[dtype])
        self.lse = torch.full((self.T, hq), MARK, device="cuda")
        self.ldq, self.ldo = ldq, ldo

    def mask_tensor(self):
        if self.words is None:
            return None
        flat = [0x123456789] * self.starts[0] + [w for ws in self.words for w in ws]
        flat += [-1] * (self.T - len(flat))
        return torch.tensor([w - (1 << 64) if w >> 63 == 1 else w for w in flat], dtype=torch.int64, device="cuda")

    def plan(self):
        cache = w4.kv_cache(self.k, self.v, self.ks, self.vs)
        cfg = w4.tree_config(self.hq, CODE[self.dtype], self.scale, self.pages.shape[1], window=self.window,
                             sinks=self.sinks, ldq=self.ldq, ldo=self.ldo)
        return cfg, cache

    def args(self):
        self.dev_pages = self.pages.cuda()
        self.dev_starts = torch.tensor(self.starts, dtype=torch.int32, device="cuda")
        self.dev_mask = self.mask_tensor()
        cfg, cache = self.plan()
        self.ws = w4.tree_workspace(cfg, cache)
        self.ws.fill_(0xFF)
        return (cfg, cache, self.q, self.dev_pages, self.lens, self.dev_starts, self.dev_mask, len(self.seqs), self.T,
                self.out, self.lse, self.ws)

    def run(self, status=0):
        w4.dec_attn_tree(*self.args())
        assert w4.w4a16_get_device_status() == status
        return self

    def want(self, b):
        """(rows, out, lse, mag, spread) of sequence b, per row [hq, d]."""
        c, n = self.seqs[b]
        seen = drafts.seen(c, n, None if self.words is None else self.words[b], self.window, self.sinks)
        j = torch.arange(c + n)
        at = (self.pages[b][j // self.page].long().cuda(), (j % self.page).cuda())
        K, V = (bits(x)[at].view(x.dtype).to(torch.float64) for x in (self.k, self.v))  # [len, hkv, d]
        if self.ks is not None:
            K, V = K * self.ks.double()[:, None], V * self.vs.double()[:, None]
        G = self.hq // self.hkv
        for i in range(n):
            row = self.starts[b] + i
            q = self.q[row, : self.hq * self.d].double().view(self.hkv, G, self.d)
            pick = torch.tensor(seen[i], dtype=torch.long, device="cuda")
            got = [drafts.attn_row(q[h], K[pick, h], V[pick, h], self.scale) for h in range(self.hkv)]
            yield (row, torch.cat([x[0] for x in got]), torch.cat([x[1] for x in got]),
                   torch.cat([x[2] for x in got]), max(x[3] for x in got))

    def check(self):
        """Every row within the rounding of its type; rows of no sequence untouched."""
        half = torch.finfo(T16[self.dtype]).eps / 2
        tiny = torch.finfo(T16[self.dtype]).smallest_normal * half
        touched = torch.zeros(self.T, dtype=torch.bool)
        for b in range(len(self.seqs)):
            for row, out, lse, mag, spread in self.want(b):
                touched[row] = True
                # scores: fp32 sums of D products; weights exact to 2^-15; numerator and denominator
                ds = spread * (self.d + 8) * 2.0 ** -24
                got = self.out[row, : self.hq * self.d].double().view(self.hq, self.d)
                bound = out.abs() * half * 1.01 + mag * (2.0 ** -14 + 2 * ds) + tiny
                bad = ~((got - out).abs() <= bound)
                assert not bool(bad.any()), (b, row, int(bad.sum()), float(((got - out).abs() / bound).nan_to_num(99).max()))
                got = self.lse[row].double()
                off = torch.where(got == lse, torch.zeros_like(lse), (got - lse).abs())
                assert bool((off <= lse.abs() * 2.0 ** -23 + ds + 2.0 ** -20).all()), (b, row, got, lse)
        assert bool((self.out[~touched] == MARK).all()) and bool((self.lse[~touched] == MARK).all())
        if self.ldo:
            assert bool((self.out[:, self.hq * self.d:] == MARK).all())
        return self


def bits(x):
    return x.view(torch.uint8) if x.dtype == torch.float8_e4m3fn else x


SMALL = [(0, 1), (37, 5), (0, 0), (300, 17), (1, 64), (129, 1), (0, 64), (255, 9)]


@pytest.mark.parametrize("dtype,kv", [("bf16", "bf16"), ("fp16", "fp16"), ("bf16", "e4m3"), ("fp16", "e4m3")])
@pytest.mark.parametrize("hq,hkv,d", [(8, 1, 128), (4, 4, 64), (6, 2, 256), (32, 2, 128), (3, 1, 96)])
def test_types_and_heads(dtype, kv, hq, hkv, d):
    Case(SMALL, hq, hkv, d, dtype, kv, pad=(2, 3), seed=hq + d).run().check()


@pytest.mark.parametrize("d", [8, 16, 24, 40, 72, 80, 136, 200, 248])
def test_head_dimensions(d):
    Case(SMALL[:5], 4, 2, d, "bf16", seed=d).run().check()
    if d % 16 == 0:
        Case(SMALL[:5], 4, 2, d, "fp16", "e4m3", seed=d).run().check()


@pytest.mark.parametrize("page", [1, 3, 5, 8, 24, 64, 100, 128, 1000])
@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_pages(page, kv):
    Case([(700, 9), (64, 64), (127, 1), (0, 3)], 8, 2, 64, "bf16", kv, page=page, seed=page).run().check()


@pytest.mark.parametrize("window,sinks", [(1, 0), (2, 1), (5, 0), (64, 4), (100, 0), (100, 130), (128, 128),
                                          (1000, 7), (30, 5000), (1 << 30, 3), (0, 9)])
@pytest.mark.parametrize("mask", ["tree", None])
def test_windows_and_sinks(window, sinks, mask):
    Case([(900, 20), (97, 64), (3, 2), (400, 1), (0, 30)], 4, 2, 64, "bf16", window=window, sinks=sinks,
         mask=mask, seed=window % 1000 + sinks).run().check()


@pytest.mark.parametrize("ctx", [0, 1, 63, 64, 65, 127, 128, 129, 255, 256, 257, 384])
def test_lengths_around_tiles(ctx):
    Case([(ctx, n) for n in (1, 2, 31, 63, 64)], 2, 1, 128, "fp16", mask=None, seed=ctx).run().check()


def test_masks_that_leave_rows_empty():
    def empty(n, rng):
        return [0 if i % 3 == 0 else (1 << n) - 1 << n | 1 << i for i in range(n)]
    # without context an empty word leaves nothing; bits from n on are ignored
    Case([(0, 7), (50, 7), (0, 40)], 4, 1, 64, "bf16", mask=empty, seed=3).run().check()
    # a window that has passed the whole context, too
    Case([(50, 7), (9, 33)], 4, 2, 64, "fp16", mask=lambda n, r: [0] * n, window=1, seed=4).run().check()


def test_random_words():
    """Any word is a mask: tokens that do not see themselves, or see later ones."""
    Case([(200, 64), (0, 64), (31, 33)], 4, 2, 64, "bf16", mask=lambda n, r: [r.getrandbits(64) for _ in range(n)],
         seed=5).run().check()


def test_strides():
    Case(SMALL, 4, 2, 64, "bf16", heads_first=True, ldq=4 * 64 + 136, ldo=4 * 64 + 8, pad=(1, 1), seed=6).run().check()
    Case(SMALL, 4, 2, 64, "fp16", "e4m3", heads_first=True, ldq=4 * 64 + 8, seed=7).run().check()


@pytest.mark.parametrize("hq,hkv", [(5, 1), (16, 1), (40, 1), (7, 7), (64, 1)])
def test_many_rows_per_head(hq, hkv):
    """Row tiles: up to 64 drafted tokens of 64 query heads are 4096 rows of one key-value head."""
    Case([(150, 64), (40, 21), (513, 1)], hq, hkv, 128, "bf16", seed=hq).run().check()


def test_large_scores_and_scales():
    Case([(500, 12)], 8, 2, 128, "bf16", spread=30.0, seed=8).run().check()
    Case([(500, 12)], 8, 2, 128, "fp16", scale=-0.3, seed=9).run().check()
    Case([(500, 12)], 8, 2, 64, "bf16", "e4m3", scale=0.0, seed=10).run().check()


def test_many_sequences():
    rng = random.Random(1)
    Case([(rng.randrange(200), rng.choice([0, 1, 1, 2, 5])) for _ in range(700)], 2, 1, 64, "bf16", seed=11).run().check()


def test_chain_is_a_tree_without_branches():
    a = Case([(300, 10), (45, 33)], 8, 2, 128, "bf16", mask=None, window=70, sinks=3, seed=12).run()
    b = Case([(300, 10), (45, 33)], 8, 2, 128, "bf16", mask=lambda n, r: w4.tree_mask(range(-1, n - 1)), window=70,
             sinks=3, seed=12).run()
    assert torch.equal(a.out, b.out) and torch.equal(a.lse, b.lse)


def test_without_lse():
    c = Case([(77, 9)], 4, 2, 64).run()
    out = torch.full_like(c.out, MARK)
    a = list(c.args())
    a[9], a[10] = out, None
    w4.dec_attn_tree(*a)
    assert torch.equal(out, c.out)


# ---- what a row does not see ----

@pytest.mark.parametrize("kv", ["bf16", "fp16", "e4m3"])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_hidden_tokens_change_nothing(kv, bad):
    """Rows that do not see a token give the same bits whatever its key and value hold: drafted tokens
    of other branches, and tokens that the window has left to some rows and not to others."""
    if kv == "e4m3" and not math.isnan(bad):
        pytest.skip("no infinities in E4M3")
    dtype = "bf16" if kv == "e4m3" else kv
    mk = lambda: Case([(300, 40), (150, 64)], 8, 2, 64, dtype, kv, window=100, sinks=2, seed=13)  # noqa: E731
    a = mk().run().check()
    for what in "kv":
        c = mk()
        for b, (ctx, n) in enumerate(c.seqs):
            for tok in (ctx + 5, ctx + n - 1, ctx - 97, ctx - 95):
                x = getattr(c, what)
                x[int(c.pages[b][tok // 16]), tok % 16] = torch.full((2, 64), bad).to(x.dtype).cuda()
        c.run()
        for b, (ctx, n) in enumerate(c.seqs):
            seen = drafts.seen(ctx, n, c.words[b], 100, 2)
            for i in range(n):
                row = c.starts[b] + i
                if not {ctx + 5, ctx + n - 1, ctx - 97, ctx - 95} & set(seen[i]):
                    assert torch.equal(a.out[row], c.out[row]) and torch.equal(a.lse[row], c.lse[row]), (what, b, i)
                elif math.isnan(bad):
                    assert bool(torch.isnan(c.out[row]).all()), (what, b, i)
                elif what == "v":
                    assert not bool(torch.isfinite(c.out[row]).any()), (what, b, i)


def test_infinite_values_and_scores():
    c = Case([(200, 9)], 4, 2, 64, "bf16", seed=14)
    at = lambda t: (int(c.pages[0][t // 16]), t % 16)  # noqa: E731
    c.v[at(100)][0, 3] = math.inf
    c.v[at(150)][0, 4] = -math.inf
    c.v[at(150)][1, 5] = math.nan
    c.v[at(203)][0, 6] = math.inf      # a drafted token's
    c.run()
    out = c.out.double().view(-1, 4, 64)
    seen = drafts.seen(200, 9, c.words[0], 0, 0)
    for row, want, lse, mag, spread in c.want(0):
        # weights here are within 2^-20 of the largest
        assert bool((out[row, :2, 3] == math.inf).all()) and bool((out[row, :2, 4] == -math.inf).all())
        assert bool(torch.isnan(out[row, 2:, 5]).all())
        drafted = out[row, :2, 6]
        assert bool((drafted == math.inf).all() if 203 in seen[row] else torch.isfinite(drafted).all())
        assert bool(torch.isfinite(out[row, 2:, 6]).all()) and bool(torch.isfinite(out[row, :, 7]).all())


def test_infinite_scores():
    c = Case([(200, 6)], 2, 2, 64, "fp16", mask=None, seed=15)
    c.q[:, 0] = 1.0
    c.k[int(c.pages[0][5]), 7][0, 0] = math.inf    # head 0: +infinity for every row
    c.q[:, 64] = 1.0
    c.k[int(c.pages[0][6]), 9][1, 0] = -math.inf   # head 1: a token of weight 0
    c.run()
    out = c.out.double().view(-1, 2, 64)
    assert bool(torch.isnan(out[:, 0]).all()) and bool((c.lse[:, 0] == math.inf).all())
    for row, want, lse, mag, spread in c.want(0):
        assert bool(((out[row, 1] - want[1]).abs() <= want[1].abs() * 2.0 ** -11 + mag[1] * 2.0 ** -12).all())


@pytest.mark.parametrize("dtype,kv", [("bf16", "bf16"), ("fp16", "fp16"), ("bf16", "e4m3")])
def test_scale_of_zero(dtype, kv):
    """All weights are alike; 0 times a query that is infinite or NaN is NaN, in its own row and head alone."""
    c = Case([(200, 6), (30, 3)], 4, 2, 64, dtype, kv, scale=0.0, seed=24)
    c.run().check()
    c.q[1, 5], c.q[7, 64 * 3 + 2] = math.inf, math.nan
    out, lse = c.out.clone(), c.lse.clone()
    c.run()
    hit = torch.zeros(c.T, 4, dtype=torch.bool, device="cuda")
    hit[1, 0] = hit[7, 3] = True
    got = c.out.view(c.T, 4, 64)
    assert bool(torch.isnan(got[hit]).all()) and bool(torch.isnan(c.lse[hit]).all())
    assert torch.equal(got[~hit], out.view(c.T, 4, 64)[~hit]) and torch.equal(c.lse[~hit], lse[~hit])


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("hq,d,page", [(8, 128, 16), (12, 64, 16), (8, 64, 5), (4, 256, 64)])
def test_signs_of_key_scales(dtype, hq, d, page):
    """Positive, negative and zero scales of neighbouring heads, in many items of one step and some of several."""
    rng = random.Random(hq + d)
    c = Case([(rng.choice([0, 3, 60, 127, 300]), rng.randrange(9)) for _ in range(180)], hq, 4, d, dtype, "e4m3", page=page,
             seed=30)
    c.ks = torch.tensor([0.05, -0.03, 0.0, 0.04], device="cuda")
    c.vs = torch.tensor([-0.05, 0.03, 0.02, 0.0], device="cuda")
    c.run().check()


def test_largest_scale():
    """Scores of 0 stay 0 under a scale whose product with log2 e is past fp32."""
    c = Case([(200, 6)], 4, 2, 64, "bf16", scale=3.0e38, seed=25)
    c.q.zero_()
    c.run().check()


def test_infinities_in_a_long_context():
    """Hidden and seen infinite values beside many tokens that all rows see."""
    c = Case([(40000, 5), (3000, 4)], 2, 1, 64, "bf16", mask=lambda n, r: [1 << i for i in range(n)], seed=26)
    want = [c.run().out.clone(), c.lse.clone()]
    for b, (ctx, n) in enumerate(c.seqs):
        c.v[int(c.pages[b][ctx // 16]), ctx % 16, 0, 9] = math.inf       # drafted token 0, seen by row 0 alone
    c.run()
    first = torch.tensor(c.starts[:-1], device="cuda")
    rest = [i for i in range(c.T) if i not in c.starts[:-1]]
    got = c.out.view(c.T, 2, 64)
    assert bool((~torch.isfinite(got[first, :, 9])).all()) and torch.equal(c.lse, want[1])
    assert torch.equal(got[rest], want[0].view(c.T, 2, 64)[rest])
    others = [d for d in range(64) if d != 9]
    assert torch.equal(got[first][..., others], want[0].view(c.T, 2, 64)[first][..., others])


@pytest.mark.parametrize("stride", ["slots", "heads"])
def test_places_that_share_memory(stride):
    """A cache whose slots, or heads, are one place in memory is read as it stands."""
    c = Case([(300, 7)], 4, 2, 64, "bf16", seed=27)
    c.k, c.v = (torch.randn(x.shape, generator=torch.Generator(device="cuda").manual_seed(s), device="cuda").to(x.dtype)
                for s, x in enumerate((c.k, c.v)))
    if stride == "slots":
        c.k, c.v = (x[:, :1].expand(-1, 16, -1, -1) for x in (c.k, c.v))
    else:
        c.k, c.v = (x[:, :, :1].expand(-1, -1, 2, -1) for x in (c.k, c.v))
    c.run().check()


def test_graphs_that_share_a_workspace():
    """Two captured calls on one workspace, replayed in turn on one stream, and an eager one between them."""
    cases = [Case([(2000, 12), (50, 3)], 8, 2, 128, "bf16", seed=28), Case([(700, 30)], 16, 2, 128, "bf16", seed=29)]
    args = [list(c.args()) for c in cases]
    args[1][-1] = args[0][-1]
    graphs = []
    for a in args:
        w4.dec_attn_tree(*a)
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            w4.dec_attn_tree(*a)
    for order in ((0, 1, 0), (1, 0, 1)):
        for c in cases:
            c.out.fill_(MARK)
        for i in order:
            graphs[i].replay()
            w4.dec_attn_tree(*args[1 - i])
        for c in cases:
            c.check()


# ---- streams, graphs, determinism ----

def test_graph_replays_with_new_lengths():
    c = Case([(300, 9), (900, 20)], 8, 2, 128, "bf16", seed=16)
    args = c.args()
    w4.dec_attn_tree(*args)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        w4.dec_attn_tree(*args)
    graph.replay()
    c.check()
    # shorter contexts, other splits of the rows: the same graph
    c.seqs = [(100, 25), (17, 4)]
    c.starts = [0, 25, 29]
    c.words = [w4.tree_mask([-1] + list(range(24))), w4.tree_mask([-1, -1, 0, 1])]
    old = c.pages.clone()
    for b, (ctx, n) in enumerate(c.seqs):
        j = torch.arange(ctx + n)
        at = (old[b][j // 16].long().cuda(), (j % 16).cuda())
        c.k[at] = torch.randn_like(c.k[at])
        c.v[at] = torch.randn_like(c.v[at])
    c.lens.copy_(torch.tensor([125, 21], dtype=torch.int32))
    c.dev_starts.copy_(torch.tensor(c.starts, dtype=torch.int32))
    c.dev_mask.copy_(c.mask_tensor())
    c.out.fill_(MARK)
    c.lse.fill_(MARK)
    graph.replay()
    c.check()
    first = c.out.clone()
    for _ in range(3):
        c.out.fill_(MARK)
        graph.replay()
        assert torch.equal(first, c.out)


def test_two_streams():
    cases = [Case([(2000, 12), (50, 3)], 8, 2, 128, "bf16", seed=s) for s in (17, 18)]
    args = [c.args() for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(5):
        for a, s in zip(args, streams):
            w4.dec_attn_tree(*a, stream=s)
    torch.cuda.synchronize()
    for c in cases:
        c.check()


def test_same_bits_every_time():
    c = Case([(5000, 30), (777, 64), (20, 1)], 16, 2, 128, "bf16", seed=19).run()
    first, lse = c.out.clone(), c.lse.clone()
    for fill in (0, 0x7F, 0xFF):
        args = c.args()
        c.ws.fill_(fill)
        w4.dec_attn_tree(*args)
        assert torch.equal(first, c.out) and torch.equal(lse, c.lse)


# ---- inputs out of range: recorded, nothing else written ----

@pytest.mark.parametrize("what", ["long", "negative", "beyond", "too_many", "descending", "short"])
def test_sequences_out_of_range(what):
    c = Case([(90, 8), (60, 12), (100, 5)], 4, 2, 64, "bf16", seed=20, pad=(0, 70))
    args = c.args()
    if what == "long":
        c.lens[1] = c.pages.shape[1] * 16 + 1
    if what == "negative":
        c.lens[1] = -1
    if what == "short":
        c.lens[1] = 11
    if what == "beyond":
        c.dev_starts[2:] = c.T + 1
    if what == "too_many":
        c.dev_starts[2:] = 8 + 65
    if what == "descending":
        c.dev_starts[2] = 3
    w4.dec_attn_tree(*args)
    assert w4.w4a16_get_device_status() == w4.W4A16_ERR_INVALID_ARG
    c.seqs = c.seqs[:1]
    got = c.out.clone(), c.lse.clone()
    first = {"descending": 3}.get(what, 8)
    assert bool((c.out[first if what == "descending" else 8: 20] == MARK).all()) or what in ("descending", "too_many")
    c.out, c.lse = got[0][: 8], got[1][: 8]
    if what != "descending":
        c.T = 8
        c.check()


def test_pages_out_of_range():
    """A page outside the cache leaves its tokens out and is recorded."""
    for page in (-1, 1 << 30, 2 ** 31 - 1):
        c = Case([(90, 8)], 4, 2, 64, "bf16", mask=None, seed=21)
        want = Case([(90, 8)], 4, 2, 64, "bf16", mask=None, seed=21)
        args = c.args()
        c.dev_pages[0, 2] = page
        w4.dec_attn_tree(*args)
        assert w4.w4a16_get_device_status() == w4.W4A16_ERR_INVALID_ARG
        j = [t for t in range(98) if not 32 <= t < 48]
        at = (want.pages[0][torch.tensor(j) // 16].long().cuda(), (torch.tensor(j) % 16).cuda())
        K, V = want.k[at].double(), want.v[at].double()
        for i in range(8):
            n = len(j) - 7 + i
            for h in range(4):
                out, lse, mag, _ = drafts.attn_row(c.q[i, 64 * h: 64 * h + 64].double()[None], K[:n, h // 2], V[:n, h // 2], c.scale)
                off = (c.out[i, 64 * h: 64 * h + 64].double() - out[0]).abs()
                assert bool((off <= out[0].abs() * 2.0 ** -8 + mag[0] * 2.0 ** -12).all())


def test_no_pages_beyond_what_is_seen():
    """Columns of the table that no row sees are not read: outside window and sinks, past the end."""
    c = Case([(900, 20)], 4, 2, 64, "bf16", window=100, sinks=20, seed=22)
    args = c.args()
    c.dev_pages[0, 3: 40] = -7          # tokens 48 .. 639: sinks and their tile stand before, the window's behind
    c.dev_pages[0, -1] = -7
    w4.dec_attn_tree(*args)
    assert w4.w4a16_get_device_status() == 0
    c.check()


def test_offsets_past_32_bits():
    """A cache whose pages lie more than 2^32 elements apart."""
    stride = (1 << 31) + 512
    k = torch.zeros(2 * stride + 16 * 64, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(23)
    kv = k.as_strided((3, 16, 1, 64), (stride, 64, 64, 1))
    kv.copy_(torch.randn(3, 16, 1, 64, generator=g, device="cuda"))
    cache = w4.kv_cache(kv, kv)
    cfg = w4.tree_config(1, w4.W4A16_BF16, 0.125, 3)
    q = torch.randn(4, 64, generator=g, device="cuda").bfloat16()
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    out = torch.empty_like(q)
    w4.dec_attn_tree(cfg, cache, q, i32(2, 0, 1), i32(40), i32(0, 4), None, 1, 4, out, None, w4.tree_workspace(cfg, cache))
    assert w4.w4a16_get_device_status() == 0
    K = torch.cat([kv[2], kv[0], kv[1]]).double()[:40, 0]
    for i in range(4):
        want, _, mag, _ = drafts.attn_row(q[i: i + 1].double(), K[: 37 + i], K[: 37 + i], 0.125)
        assert bool(((out[i].double() - want[0]).abs() <= want[0].abs() * 2.0 ** -8 + mag[0] * 2.0 ** -12).all())


def test_agrees_with_single_token_attention():
    """One drafted token is what dec_attn_paged computes."""
    c = Case([(n, 1) for n in (0, 5, 127, 1000, 2500)], 16, 2, 128, "bf16", mask=None, window=600, seed=24).run().check()
    cfg, cache = c.plan()
    one = w4.attn_config(16, w4.W4A16_BF16, c.scale, c.pages.shape[1], window=600)
    out, lse = torch.empty_like(c.out), torch.empty_like(c.lse)
    w4.dec_attn_paged(one, cache, c.q, c.dev_pages, c.lens, 5, out, lse, w4.attn_workspace(one, cache))
    assert w4.w4a16_get_device_status() == 0
    # each within the rounding of exact: half a step and 2^-13 of the magnitude each
    mag = torch.cat([m for b in range(5) for _, _, _, m, _ in c.want(b)]).view(5, -1)
    assert bool(((out.double() - c.out.double()).abs() <= out.double().abs() * 2.0 ** -7 + mag * 2.0 ** -11).all())
    assert bool(((lse - c.lse).abs() <= lse.abs() * 2.0 ** -21 + 2.0 ** -12).all())
