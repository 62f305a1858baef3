"""A decoding loop with drafted trees: append, attention of the tree, log probabilities, the accepted path
moved to the context's end, and the next step over it; beside a plain 64-bit account of the same loop."""
import random

import pytest
import torch

import weight_only_int4_tma_gb300 as w4
from oracle import drafts
from oracle import layer as ol

pytestmark = pytest.mark.gpu

HQ, HKV, D, PAGE, COLS, VOCAB = 8, 2, 64, 16, 20, 1000
KV = {"bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}


def bits(x):
    return x.view(torch.uint8) if x.dtype == torch.float8_e4m3fn else x.view(torch.int16)


class Loop:
    def __init__(self, kv, n, window=0, sinks=0):
        self.g, self.rng = torch.Generator(device="cuda").manual_seed(n), random.Random(n)
        self.ctx, self.n, self.window, self.sinks = [0, 37, 200], n, window, sinks
        B, T = len(self.ctx), len(self.ctx) * n
        self.B, self.T, self.H = B, T, (HQ + 2 * HKV) * D
        self.embed = self.randn(VOCAB, self.H)
        self.unembed = self.randn(HQ * D, VOCAB) * 0.25
        self.table = torch.empty(COLS * PAGE, D, device="cuda")
        w4.dec_rope_table(D, 10000.0, None, self.table, COLS * PAGE)
        self.k, self.v = (bits(self.randn(B * COLS, PAGE, HKV, D).to(KV[kv])).clone().view(KV[kv]) for _ in range(2))
        self.scales = [0.5 + torch.rand(HKV, generator=self.g, device="cuda") for _ in range(2)] if kv == "e4m3" else [None, None]
        self.cache = w4.kv_cache(self.k, self.v, *self.scales)
        self.pages = torch.randperm(B * COLS, generator=self.g, device="cuda").view(B, COLS).int()
        self.rc = w4.rope_config(HQ, HKV, D, w4.W4A16_BF16, self.table, D, ldq=self.H, ldk=self.H, ldv=self.H)
        self.tc = w4.tree_config(HQ, w4.W4A16_BF16, D ** -0.5, COLS, window=window, sinks=sinks)
        self.lc = w4.logprob_config(VOCAB, w4.DEC_LOGITS_BF16, n_ids=n, top=1)
        self.ws = w4.tree_workspace(self.tc, self.cache)
        new = lambda *s, t=torch.int32: torch.zeros(*s, dtype=t, device="cuda")  # noqa: E731
        self.x, self.q, self.out = (new(T, w, t=torch.bfloat16) for w in (self.H, HQ * D, HQ * D))
        self.pos, self.slots, self.mask = new(T), new(T, t=torch.int64), new(T, t=torch.int64)
        self.lens, self.starts = new(B), torch.arange(B + 1, device="cuda").int() * n
        self.ids, self.logprobs = new(T, n), new(T, n, t=torch.float32)
        self.lse, self.entropy, self.best, self.best_lp = new(T, t=torch.float32), new(T, t=torch.float32), new(T, 1), new(T, 1, t=torch.float32)
        self.src, self.dst, self.groups = new(T, t=torch.int64), new(T, t=torch.int64), new(B + 1)
        self.history = [[bits(x)[at].clone() for x in (self.k, self.v)]
                        for at in (self.places(b, range(c)) for b, c in enumerate(self.ctx))]

    def randn(self, *s):
        return torch.randn(*s, generator=self.g, device="cuda").to(torch.bfloat16)

    def places(self, b, tokens):
        j = torch.tensor(list(tokens), dtype=torch.long, device="cuda")
        return self.pages[b][j // PAGE].long(), j % PAGE

    def slot(self, b, j):
        return int(self.pages[b][j // PAGE]) * PAGE + j % PAGE

    def draft(self):
        """New trees of n tokens behind every context."""
        self.parents, pos, slots, mask, tokens = [], [], [], [], []
        ids = torch.full((self.T, self.n), -1, dtype=torch.int32)
        for b in range(self.B):
            par = [-1] + [self.rng.randrange(i) for i in range(1, self.n)]
            tok = [self.rng.randrange(VOCAB) for _ in par]
            depth = []
            for i, p in enumerate(par):
                depth.append(depth[p] + 1 if p >= 0 else 0)
                if p >= 0:
                    ids[b * self.n + p, i] = tok[i]       # the children's tokens, each in its own column
            self.parents.append(par)
            pos += [self.ctx[b] + x for x in depth]
            slots += [self.slot(b, self.ctx[b] + i) for i in range(self.n)]
            mask += w4.tree_mask(par)
            tokens += tok
        self.depth = [p - self.ctx[i // self.n] for i, p in enumerate(pos)]
        for to, value in ((self.pos, pos), (self.slots, slots), (self.mask, mask),
                          (self.lens, [c + self.n for c in self.ctx])):
            to.copy_(torch.tensor(value, dtype=to.dtype))
        self.ids.copy_(ids)
        self.x.copy_(self.embed[torch.tensor(tokens, device="cuda")])

    def step(self):
        x = self.x
        w4.dec_rope_append(self.rc, self.cache, x, x[:, HQ * D:], x[:, (HQ + HKV) * D:], self.T, self.pos, self.slots, self.q)
        w4.dec_attn_tree(self.tc, self.cache, self.q, self.pages, self.lens, self.starts, self.mask, self.B, self.T,
                         self.out, None, self.ws)
        self.logits = self.out @ self.unembed
        w4.dec_token_logprobs(self.lc, self.logits, None, self.ids, self.T, self.logprobs, self.lse, self.entropy,
                              self.best, self.best_lp)

    def near(self, got, q, K, V):
        """One row's attention within its rounding (the bounds of the attention's own tests)."""
        bad = False
        for h in range(HKV):
            rows = slice(h * (HQ // HKV), (h + 1) * (HQ // HKV))
            k, v = (x[:, h].view(x.dtype).double() * (1.0 if s is None else s[h].double()) for x, s in ((K, self.scales[0]), (V, self.scales[1])))
            out, _, mag, spread = drafts.attn_row(q.view(HQ, D)[rows].double(), k, v, D ** -0.5)
            bound = out.abs() * 2.0 ** -8 * 1.01 + mag * (2.0 ** -14 + 2 * spread * (D + 8) * 2.0 ** -24) + 2.0 ** -130
            bad |= bool(((got.view(HQ, D)[rows].double() - out).abs() > bound).any())
        return not bad

    def check_and_accept(self):
        src, dst, groups = [], [], [0]
        want = torch.log_softmax(self.logits.double(), 1)
        assert torch.equal(self.logits.gather(1, self.best.long()), self.logits.max(1, keepdim=True).values)
        for b in range(self.B):
            ctx, n = self.ctx[b], self.n
            new = [bits(x)[self.places(b, range(ctx, ctx + n))].clone() for x in (self.k, self.v)]
            rows = slice(b * n, (b + 1) * n)
            if self.k.dtype == torch.bfloat16:
                key, _ = ol.rope(self.x[rows, HQ * D:(HQ + HKV) * D].reshape(n, HKV, D), self.table[self.pos[rows].long()], D, False)
                assert float((new[0].view(torch.bfloat16).double() - key).abs().max()) <= 2.0 ** -7 * float(key.abs().max())
                assert torch.equal(new[1].view(torch.bfloat16), self.x[rows, (HQ + HKV) * D:].reshape(n, HKV, D))
            for i in range(n):
                path, j = [], i
                while j >= 0:
                    path.insert(0, j)
                    j = self.parents[b][j]
                depth = len(path)
                old = [j for j in range(ctx) if self.window == 0 or j < self.sinks or j >= ctx + depth - self.window]
                K, V = (torch.cat([h[old], x[path]]).view(self.k.dtype) for h, x in zip(self.history[b], new))
                assert self.near(self.out[b * n + i], self.q[b * n + i], K, V), (b, i)
                for c in range(n):
                    if self.parents[b][c] == i:
                        got, exact = float(self.logprobs[b * n + i, c]), float(want[b * n + i, int(self.ids[b * n + i, c])])
                        assert abs(got - exact) <= 2.0 ** -20 * max(1.0, abs(exact)) + 2.0 ** -22 * float(self.lse[b * n + i].abs()), (b, i, c)
            # the accepted path: from the root to the likelier child, down to some depth
            path, stop = [0], self.rng.randrange(n)
            while len(path) <= stop:
                row = b * n + path[-1]
                kids = [c for c in range(n) if self.parents[b][c] == path[-1]]
                if not kids:
                    break
                path.append(max(kids, key=lambda c: float(self.logprobs[row, c])))
            src += [self.slot(b, ctx + i) for i in path]
            dst += [self.slot(b, ctx + i) for i in range(len(path))]
            groups.append(len(src))
            self.history[b] = [torch.cat([h, x[path]]) for h, x in zip(self.history[b], new)]
            self.ctx[b] = ctx + len(path)
        for to, value in ((self.src, src), (self.dst, dst), (self.groups, groups)):
            to[: len(value)].copy_(torch.tensor(value, dtype=to.dtype))

    def close_up(self):
        w4.dec_kv_move(self.cache, self.src, self.dst, self.groups, self.B, self.T)

    def check_cache(self):
        for b in range(self.B):
            for x, want in zip((self.k, self.v), self.history[b]):
                assert torch.equal(bits(x)[self.places(b, range(self.ctx[b]))], want), b


@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("kv,n,window,sinks", [("bf16", 12, 0, 0), ("e4m3", 9, 0, 0), ("bf16", 24, 48, 3), ("e4m3", 1, 0, 0)])
def test_drafting_loop(kv, n, window, sinks, graph):
    loop = Loop(kv, n, window, sinks)
    step, close_up = loop.step, loop.close_up
    if graph:
        loop.draft()
        loop.step()     # (writes only slots behind the contexts)
        loop.close_up()  # (empty groups)
        torch.cuda.synchronize()
        a, z = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
        with torch.cuda.graph(a):
            loop.step()
        with torch.cuda.graph(z):
            loop.close_up()
        step, close_up = a.replay, z.replay
    for _ in range(4):
        loop.draft()
        step()
        loop.check_and_accept()
        close_up()
        assert w4.w4a16_get_device_status() == 0
        loop.check_cache()
    # and the one-token operator reads the same context
    q, out = loop.randn(loop.B, HQ * D), loop.randn(loop.B, HQ * D)
    lens = torch.tensor(loop.ctx, dtype=torch.int32, device="cuda")
    ac = w4.attn_config(HQ, w4.W4A16_BF16, D ** -0.5, COLS)
    w4.dec_attn_paged(ac, loop.cache, q, loop.pages, lens, loop.B, out, None, w4.attn_workspace(ac, loop.cache))
    assert w4.w4a16_get_device_status() == 0
    for b in range(loop.B):
        K, V = (h.view(loop.k.dtype) for h in loop.history[b])
        assert loop.near(out[b], q[b], K, V), b
