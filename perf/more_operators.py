"""Operators of speculative decoding on real work: cases, plain forms and exact values.

A serving program that has several tokens drafted per sequence runs three operators around the
4-bit GEMMs and the decoder-layer operators of this library:

* tree: attention of up to 64 drafted tokens per sequence, in a tree or a chain, over the paged
  cache (fp16, bf16 or E4M3 with a scale per head) that already holds their keys and values; with
  a sliding window and first tokens that stay visible where asked for;
* logprob: log-sum-exp and entropy of every row of logits, the log probabilities of given tokens
  and the largest logits with theirs;
* move: the accepted tokens' keys and values moved to the slots right behind the context.

With ``own`` false, ``run`` computes them with elementary torch operations in 32 bits, rounded
once at the end; with ``own`` true it makes the library's calls.  ``exact`` states the same
definitions in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32, "e4m3": torch.float8_e4m3fn}
BYTES = {"fp16": 2, "bf16": 2, "fp32": 4, "e4m3": 1}


def _tree(b, n, ragged, context, q_heads, kv_heads, d, dtype, kv, page, window=0, sinks=0, chain=False,
          lse=False, pad=0, name=None):
    c = {"op": "tree", "b": b, "n": n, "ragged": ragged, "context": context, "q_heads": q_heads,
         "kv_heads": kv_heads, "d": d, "dtype": dtype, "kv": kv, "page": page, "window": window,
         "sinks": sinks, "chain": chain, "lse": lse, "pad": pad}
    return dict(c, name=name) if name else c


def _logprob(t, vocab, dtype, ids, top, temperature, name=None):
    c = {"op": "logprob", "t": t, "vocab": vocab, "dtype": dtype, "ids": ids, "top": top,
         "temperature": temperature}
    return dict(c, name=name) if name else c


def _move(b, most, kv_heads, d, kv, page, heads_first, name=None):
    c = {"op": "move", "b": b, "most": most, "kv_heads": kv_heads, "d": d, "kv": kv, "page": page,
         "heads_first": heads_first}
    return dict(c, name=name) if name else c


def listed():
    return [
        # a single short conversation, a small tree: latency counts
        _tree(1, 8, False, 777, 64, 8, 128, "bf16", "bf16", 64, name="tree_b1_n8_l777"),
        # a ragged batch with a key-value head for each query head, idle slots, padded rows
        _tree(16, 16, True, 4096, 32, 32, 128, "fp16", "fp16", 16, lse=True, pad=13, name="tree_heads32_b16"),
        # one long document and the largest tree: 512 rows for each key-value head
        _tree(1, 64, False, 32768, 64, 8, 128, "bf16", "bf16", 64, name="tree_b1_n64_l32768"),
        # a full serving batch with trees of up to 32 tokens
        _tree(32, 32, True, 8192, 64, 8, 128, "bf16", "bf16", 64, name="tree_b32_n32_l8192"),
        # 8-bit cache, narrow heads, a window with four sinks over longer sequences
        _tree(33, 12, True, 9000, 32, 4, 64, "bf16", "e4m3", 32, window=4096, sinks=4, name="tree_e4m3_window"),
        # single tokens with a window and a page of sinks: an endless conversation's step
        _tree(48, 1, False, 20000, 64, 8, 128, "bf16", "bf16", 64, window=2048, sinks=64, chain=True,
              name="sinks_b48_n1"),
        # one row of logits of a large vocabulary: a single stream's step
        _logprob(1, 128000, "bf16", 1, 5, False, name="logprob_t1_v128000"),
        # a tree's rows: candidates of each node, twenty alternatives, temperatures per request
        _logprob(60, 32000, "fp16", 4, 20, True, name="logprob_t60_v32000"),
        # scoring a prompt: one given token per row, no alternatives
        _logprob(2048, 128000, "bf16", 1, 0, False, name="logprob_t2048_v128000"),
        # an odd batch of 32-bit logits, rows that are not 16-byte aligned
        _logprob(301, 50001, "fp32", 1, 20, True, name="logprob_t301_v50001"),
        # one sequence's accepted path, all that a single stream moves
        _move(1, 4, 8, 128, "bf16", 64, False, name="move_b1"),
        # a large batch, pages that hold heads of all tokens
        _move(256, 12, 8, 128, "fp16", 16, True, name="move_b256"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tree", "tree", "tree", "logprob", "logprob", "move"])
    if op == "logprob":
        vocab = _log(rng, 1000, 260000)
        vocab = vocab if rng.random() < 0.4 else vocab // 8 * 8
        t = _log(rng, 1, min(4096, 2048 * 128000 // 2 // vocab))
        return _logprob(t, vocab, rng.choice(["fp16", "bf16", "fp32"]), rng.choice([0, 1, 1, rng.randint(2, 16)]),
                        rng.choice([0, 1, 5, 20, rng.randint(1, 32)]), rng.random() < 0.5)
    dtype = rng.choice(["fp16", "bf16"])
    kv = rng.choice([dtype, dtype, "e4m3"])
    d = rng.choice([64, 64, 80, 96, 128, 128, 128, 256])
    kv_heads = rng.choice([1, 2, 4, 8, 8, 16, 32])
    page = rng.choice([1, 5, 8, 16, 16, 24, 32, 64, 64, 128, 256])
    if op == "move":
        return _move(_log(rng, 1, 256), rng.randint(1, 16), kv_heads, d, kv, page, rng.random() < 0.5)
    q_heads = kv_heads * rng.choice([g for g in (1, 2, 3, 4, 7, 8, 12, 16) if g * kv_heads <= 128])
    b = _log(rng, 1, 64)
    n = _log(rng, 1, 64)
    # half of what the largest listed cases hold and score, so that none costs more
    most = min(32 * 8192 * 8 * 128 // 2 // (b * kv_heads * d), 64 * 64 * 32768 * 128 // 2 // (b * q_heads * n * d))
    context = _log(rng, 1, max(2, min(131072, most)))
    window = rng.choice([0, 0, 0, _log(rng, 16, 8192)])
    return _tree(b, n, rng.random() < 0.7, context, q_heads, kv_heads, d, dtype, kv, page, window,
                 rng.choice([0, 1, 4, _log(rng, 1, 300)]) if window else 0, rng.random() < 0.3,
                 rng.random() < 0.4, rng.choice([0, 0, rng.randint(1, 20)]))


def _spread(i):
    """The golden ratio's multiples: from 1 down, well spread over 0 .. 1."""
    return (1.0 - i * 0.6180339887498949) % 1.0 if i else 1.0


def _sequences(case):
    """(context, drafted tokens) of every sequence, up to their order: all alike, or spread from a
    tenth of the longest to the longest, with one in five that has nothing drafted."""
    got = []
    for i in range(case["b"]):
        if not case["ragged"]:
            got.append((case["context"], case["n"]))
            continue
        context = max(1, int(case["context"] * (0.1 + 0.9 * _spread(i))))
        got.append((context, 0 if i % 5 == 4 else max(1, int(case["n"] * (0.3 + 0.7 * _spread(i + 7))))))
    return got


def _moved(case):
    """How many tokens each sequence moves."""
    return [max(1, int(case["most"] * _spread(i))) if i % 6 != 5 else 0 for i in range(case["b"])]


def work(case):
    if case["op"] == "logprob":
        t, v, e = case["t"], case["vocab"], BYTES[case["dtype"]]
        moved = t * v * e + t * (8 + 8 * case["ids"] + 8 * case["top"] + (4 if case["temperature"] else 0))
        return {"bytes": moved, "flops": 5 * t * v}
    d, hkv = case["d"], case["kv_heads"]
    row = 2 * hkv * d * BYTES[case["kv"]]  # a cached token's keys and values
    if case["op"] == "move":
        moved = sum(_moved(case))
        return {"bytes": moved * (2 * row + 16) + 4 * case["b"], "flops": 0}
    hq, moved, flops = case["q_heads"], 0, 0
    for context, n in _sequences(case):
        if not n:
            continue
        read = context
        if case["window"]:
            read = min(context, case["sinks"] + case["window"] - 1)
        moved += (read + n) * row + 4 * n * hq * d + 8 * n + 4 * (-(-(read + n) // case["page"]) + 2)
        moved += 4 * n * hq if case["lse"] else 0
        # about half of the drafted tokens of a chain are ancestors, fewer in a tree
        flops += 4 * d * hq * n * (read + (n + 1) // 2)
    return {"bytes": max(moved, 1), "flops": flops}


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(shape, dtype, g, scale=1.0):
    wide = torch.float16 if dtype == torch.float8_e4m3fn else dtype
    return torch.randn(shape, generator=g, device="cuda", dtype=wide).mul_(scale).to(dtype)


def _pages(count, page, heads, d, kv, g, heads_first=False):
    """A cache's key or value pages as a model leaves them: unit normal values (8-bit caches hold
    them over the head's scale); in memory tokens of all heads, or heads of all tokens."""
    shape = (count, heads, page, d) if heads_first else (count, page, heads, d)
    x = _normal(shape, DTYPES[kv], g, 16.0 if kv == "e4m3" else 1.0)
    return x.transpose(1, 2) if heads_first else x


def _bits(x):
    return x.view(torch.uint8) if x.dtype == torch.float8_e4m3fn else x


def _ancestors(parents):
    """For each token of a tree the bits of the tokens it sees: its ancestors and itself."""
    bits = []
    for i, p in enumerate(parents):
        bits.append((bits[p] if p >= 0 else 0) | 1 << i)
    return [v - (1 << 64) if v >> 63 else v for v in bits]


def prepare(case, seed):
    g = _gen(seed)
    s = {"case": case}
    if own:
        import weight_only_int4_tma_gb300 as w4
        s["w4"] = w4
    {"tree": _prepare_tree, "logprob": _prepare_logprob, "move": _prepare_move}[case["op"]](s, case, g)
    return s


def _prepare_tree(s, c, g):
    dtype, d, hq, hkv, page, b = DTYPES[c["dtype"]], c["d"], c["q_heads"], c["kv_heads"], c["page"], c["b"]
    order = torch.randperm(b, generator=g, device="cuda").tolist()
    sequences = [_sequences(c)[i] for i in order]
    counts = [n for _, n in sequences]
    lens = [context + n for context, n in sequences]
    starts = [0]
    for n in counts:
        starts.append(starts[-1] + n)
    t = starts[-1] + c["pad"]  # rows behind the last sequence: a captured batch's padding
    s["t"], s["longest"], s["drafted"] = t, max(lens), max(counts)
    s["starts"] = torch.tensor(starts, dtype=torch.int32, device="cuda")
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    columns = -(-max(lens) // page)
    count = b * columns + 1
    s["q"] = _normal((t, hq * d), dtype, g, 1.5)
    s["k"], s["v"] = (_pages(count, page, hkv, d, c["kv"], g) for _ in range(2))
    s["pages"] = torch.randperm(count, generator=g, device="cuda")[: b * columns].view(b, columns).int()
    # what lies in a page past a sequence's end is left from another one: any bits
    length = s["lens"].long()
    at = s["pages"].long().gather(1, (length // page).clamp(max=columns - 1)[:, None]).squeeze(1)
    stale = (torch.arange(page, device="cuda") >= (length % page)[:, None]) & (length % page != 0)[:, None]
    for x in (s["k"], s["v"]):
        bits = x.view(torch.uint8 if c["kv"] == "e4m3" else torch.int16)
        bits[at] = bits[at].masked_fill(stale[:, :, None, None], 0x7F if c["kv"] == "e4m3" else 0x7FFF)
    s["mask"] = None
    if not c["chain"]:  # trees in draft order: every token's parent is one of the eight before it
        back = torch.rand(64 * b, generator=g, device="cuda").tolist()
        bits = []
        for i, n in enumerate(counts):
            bits += _ancestors([j - 1 - int(back[64 * i + j] * min(j, 8)) for j in range(n)])
        s["mask"] = torch.tensor(bits + [0] * c["pad"], dtype=torch.int64, device="cuda")
    s["out"] = torch.zeros((t, hq * d), dtype=dtype, device="cuda")
    s["lse"] = torch.zeros((t, hq), dtype=torch.float32, device="cuda") if c["lse"] else None
    # 8-bit caches: the value of a stored number is the number times its head's scale
    s["k_scale"], s["v_scale"] = ((0.05 + 0.02 * torch.rand(hkv, generator=g, device="cuda"))
                                  if c["kv"] == "e4m3" else None for _ in range(2))
    if own:  # the handles that a serving program keeps: cache, settings, workspace
        w4 = s["w4"]
        code = w4.W4A16_FP16 if c["dtype"] == "fp16" else w4.W4A16_BF16
        s["cache"] = w4.kv_cache(s["k"], s["v"], s["k_scale"], s["v_scale"])
        s["plan"] = w4.tree_config(hq, code, d ** -0.5, columns, window=c["window"], sinks=c["sinks"])
        s["workspace"] = w4.tree_workspace(s["plan"], s["cache"])


def _prepare_logprob(s, c, g):
    t, v, dtype = c["t"], c["vocab"], DTYPES[c["dtype"]]
    # logits as a trained model's head gives them: a broad body and a few tokens that stand out
    x = torch.empty((t, v), dtype=dtype, device="cuda")
    for r in range(0, t, 256):
        rows = torch.randn((min(256, t - r), v), generator=g, device="cuda").mul_(2.5)
        at = torch.randint(0, v, (rows.shape[0], 12), generator=g, device="cuda")
        rows.scatter_add_(1, at, 14.0 * torch.rand(at.shape, generator=g, device="cuda"))
        x[r: r + 256] = rows.to(dtype)
    s["x"] = x
    s["factor"] = 0.5 + torch.rand(t, generator=g, device="cuda") if c["temperature"] else None
    s["ids"] = torch.randint(0, v, (t, c["ids"]), generator=g, device="cuda").int() if c["ids"] else None
    new = lambda n, kind: torch.empty((t, n), dtype=kind, device="cuda") if n else None  # noqa: E731
    s["logprobs"], s["top_ids"] = new(c["ids"], torch.float32), new(c["top"], torch.int32)
    s["top_logprobs"] = new(c["top"], torch.float32)
    s["lse"], s["entropy"] = (torch.empty(t, device="cuda") for _ in range(2))
    if own:
        w4 = s["w4"]
        kind = {"fp16": w4.DEC_LOGITS_FP16, "bf16": w4.DEC_LOGITS_BF16, "fp32": w4.DEC_LOGITS_FP32}[c["dtype"]]
        s["plan"] = w4.logprob_config(v, kind, n_ids=c["ids"], top=c["top"])


def _prepare_move(s, c, g):
    """Every sequence has its context in pages of its own and 64 slots of drafted tokens behind it;
    the accepted ones are spread over those and move to the first."""
    b, page = c["b"], c["page"]
    context = torch.randint(1, 200, (b,), generator=g, device="cuda").tolist()
    columns = -(-(200 + 64) // page)
    count = b * columns
    s["k"], s["v"] = (_pages(count, page, c["kv_heads"], c["d"], c["kv"], g, c["heads_first"]) for _ in range(2))
    table = torch.randperm(count, generator=g, device="cuda").view(b, columns).tolist()
    slot = lambda i, j: table[i][j // page] * page + j % page  # noqa: E731
    pick = torch.rand(b, 16, generator=g, device="cuda").tolist()
    src, dst, starts = [], [], [0]
    for i, n in enumerate(_moved(c)):
        at = 16  # breadth first: the path's tokens stand behind the slots that they move to
        for j in range(n):
            at += 1 + int(2.9 * pick[i][j])
            src.append(slot(i, context[i] + at))
            dst.append(slot(i, context[i] + j))
        starts.append(len(src))
    s["src"], s["dst"] = (torch.tensor(x, dtype=torch.int64, device="cuda") for x in (src, dst))
    s["starts"] = torch.tensor(starts, dtype=torch.int32, device="cuda")
    if own:
        s["cache"] = s["w4"].kv_cache(s["k"], s["v"])


def run(state):
    return {"tree": _run_tree, "logprob": _run_logprob, "move": _run_move}[state["case"]["op"]](state)


def _run_tree(s):
    c = s["case"]
    if own:
        s["w4"].dec_attn_tree(s["plan"], s["cache"], s["q"], s["pages"], s["lens"], s["starts"], s["mask"], c["b"],
                              s["t"], s["out"], s["lse"], s["workspace"])
        return {"out": s["out"], "lse": s["lse"]}
    b, d, hq, hkv, n = c["b"], c["d"], c["q_heads"], c["kv_heads"], s["drafted"]
    pages = s["pages"].long()

    def cached(x, scale):  # [b, kv heads, tokens, d] in 32 bits
        x = _bits(x)[pages].view(x.dtype).flatten(1, 2)[:, : s["longest"]].transpose(1, 2).float()
        return x if scale is None else x * scale[:, None, None]

    k, v = cached(s["k"], s["k_scale"]), cached(s["v"], s["v_scale"])
    starts, lens = s["starts"].long(), s["lens"].long()
    count = starts[1:] - starts[:-1]
    i = torch.arange(n, device=k.device)
    live = i < count[:, None]                                       # [b, n]
    rows = torch.where(live, starts[:-1, None] + i, s["t"])         # a row of their own for the others
    at = torch.arange(k.shape[2], device=k.device)
    context = (lens - count)[:, None, None]
    j = at - context                                                # [b, 1, tokens], of the drafted ones
    if s["mask"] is None:
        depth = (i + 1).expand(b, n)
        drafted = j <= i[:, None]
    else:
        word = torch.cat([s["mask"], s["mask"].new_zeros(1)])[rows]  # [b, n]
        depth = (word[..., None] >> torch.arange(64, device=k.device) & 1).sum(2)
        drafted = (word[..., None] >> j.clamp(0, 63) & 1) == 1
    seen = at < context
    if c["window"]:
        seen = seen & ((at < c["sinks"]) | (at >= context + depth[..., None] - c["window"]))
    seen = torch.where(j < 0, seen, drafted) & (at < lens[:, None, None]) & live[..., None]
    seen = seen[:, None, :, None, :]                                # [b, 1, n, 1, tokens]
    q = torch.cat([s["q"], s["q"].new_zeros((1, hq * d))])[rows].float()
    q = q.view(b, n, hkv, hq // hkv, d).transpose(1, 2).reshape(b, hkv, -1, d)
    score = (torch.matmul(q, k.transpose(2, 3)) * d ** -0.5).view(b, hkv, n, hq // hkv, -1)
    score = score.masked_fill_(~seen, -math.inf)
    most = score.amax(4, keepdim=True)
    p = score.sub_(most.masked_fill(most == -math.inf, 0.0)).exp_()
    total = p.sum(4, keepdim=True)
    v = v.masked_fill((at >= lens[:, None])[:, None, :, None], 0.0)
    out = torch.matmul(p.flatten(2, 3), v).view(b, hkv, n, hq // hkv, d) / total.masked_fill(total == 0, 1.0)
    out = out.transpose(1, 2).reshape(b * n, hq * d).to(s["q"].dtype)
    result = torch.cat([s["out"], s["out"].new_zeros((1, hq * d))])
    result[rows.flatten()] = out
    lse = None
    if c["lse"]:
        lse = torch.cat([s["lse"], s["lse"].new_zeros((1, hq))])
        lse[rows.flatten()] = (most + total.log()).squeeze(4).transpose(1, 2).reshape(b * n, hq)
        lse = lse[: s["t"]]
    return {"out": result[: s["t"]], "lse": lse}


def _run_logprob(s):
    c = s["case"]
    if own:
        s["w4"].dec_token_logprobs(s["plan"], s["x"], s["factor"], s["ids"], c["t"], s["logprobs"], s["lse"],
                                   s["entropy"], s["top_ids"], s["top_logprobs"])
        return {"logprobs": s["logprobs"], "lse": s["lse"], "entropy": s["entropy"], "top_ids": s["top_ids"],
                "top_logprobs": s["top_logprobs"]}
    z = s["x"].float()
    if s["factor"] is not None:
        z = z * s["factor"][:, None]
    most = z.amax(1, keepdim=True)
    e = torch.exp(z - most)
    total = e.sum(1, dtype=torch.float64)
    lse = most.squeeze(1).double() + total.log()
    entropy = total.log() - (e * (z - most)).sum(1, dtype=torch.float64) / total
    got = {"logprobs": None, "lse": lse.float(), "entropy": entropy.float(), "top_ids": None, "top_logprobs": None}
    if c["ids"]:
        got["logprobs"] = (z.gather(1, s["ids"].long()).double() - lse[:, None]).float()
    if c["top"]:
        # the lowest index of the largest, one after another
        rest, ids = s["x"].float(), []
        for _ in range(c["top"]):
            at = rest.eq(rest.amax(1, keepdim=True)).int().argmax(1, keepdim=True)
            ids.append(at)
            rest = rest.scatter(1, at, -math.inf)
        ids = torch.cat(ids, 1)
        got["top_ids"] = ids.int()
        got["top_logprobs"] = (z.gather(1, ids).double() - lse[:, None]).float()
    return got


def _run_move(s):
    c = s["case"]
    if own:
        s["w4"].dec_kv_move(s["cache"], s["src"], s["dst"], s["starts"], c["b"], s["src"].numel())
        return {"k": s["k"], "v": s["v"]}
    for x in (s["k"], s["v"]):
        x = _bits(x)
        src, dst = s["src"], s["dst"]
        x[dst // c["page"], dst % c["page"]] = x[src // c["page"], src % c["page"]]
    return {"k": s["k"], "v": s["v"]}


def exact(case, seed):
    """What run() returns, from the operators' definitions in 64 bits."""
    s = prepare(case, seed)
    return {"tree": _exact_tree, "logprob": _exact_logprob, "move": _exact_move}[case["op"]](s, case)


def _exact_tree(s, c):
    f64, d, hq, hkv, page = torch.float64, c["d"], c["q_heads"], c["kv_heads"], c["page"]
    group = hq // hkv
    out = s["out"].to(f64).view(-1, hq, d).clone()
    lse = s["lse"].to(f64).clone() if c["lse"] else None
    starts, words = s["starts"].tolist(), None if s["mask"] is None else s["mask"].tolist()
    for b, length in enumerate(s["lens"].tolist()):
        first, last = starts[b], starts[b + 1]
        if first == last:
            continue
        context = length - (last - first)
        hidden = torch.zeros((last - first, length), dtype=torch.bool)
        for i in range(last - first):
            sees = [j for j in range(last - first) if (j <= i if words is None else words[first + i] >> j & 1)]
            if c["window"]:
                hidden[i, c["sinks"]: max(c["sinks"], context + len(sees) - c["window"])] = True
            hidden[i, context:] = True
            hidden[i, [context + j for j in sees]] = False
        hidden = hidden.to(s["q"].device)
        slot = torch.arange(length, device=s["q"].device)
        page_of = s["pages"][b].long()[slot // page]
        for h in range(hkv):
            k, v = (_bits(s[x])[page_of, slot % page, h].view(s[x].dtype).to(f64) for x in ("k", "v"))
            if c["kv"] == "e4m3":
                k, v = k * s["k_scale"][h].to(f64), v * s["v_scale"][h].to(f64)
            q = s["q"][first:last].to(f64).view(-1, hq, d)[:, h * group: (h + 1) * group]
            score = torch.einsum("igd,td->igt", q, k) / math.sqrt(d)
            score = torch.where(hidden[:, None, :], torch.full_like(score, -math.inf), score)
            p = torch.softmax(score, 2)
            out[first:last, h * group: (h + 1) * group] = torch.einsum("igt,td->igd", p, v)
            if c["lse"]:
                lse[first:last, h * group: (h + 1) * group] = torch.logsumexp(score, 2)
    return {"out": out.view(-1, hq * d), "lse": lse}


def _exact_logprob(s, c):
    got = {"logprobs": [], "lse": [], "entropy": [], "top_ids": [], "top_logprobs": []}
    for r in range(0, c["t"], 128):
        x = s["x"][r: r + 128].to(torch.float64)
        z = x if s["factor"] is None else x * s["factor"][r: r + 128].to(torch.float64)[:, None]
        logp = torch.log_softmax(z, 1)
        got["lse"].append(torch.logsumexp(z, 1))
        got["entropy"].append(-(logp.exp() * logp).sum(1))
        if c["ids"]:
            got["logprobs"].append(logp.gather(1, s["ids"][r: r + 128].long()))
        if c["top"]:
            at = torch.sort(x, dim=1, descending=True, stable=True).indices[:, : c["top"]]
            got["top_ids"].append(at.int())
            got["top_logprobs"].append(logp.gather(1, at))
    return {name: torch.cat(parts) if parts else None for name, parts in got.items()}


def _exact_move(s, c):
    got = {}
    for name in ("k", "v"):
        x = s[name].to(torch.float64).transpose(0, 1).contiguous().transpose(0, 1)
        for a, b in zip(s["src"].tolist(), s["dst"].tolist()):
            x[b // c["page"], b % c["page"]] = x[a // c["page"], a % c["page"]].clone()
        got[name] = x
    return got
