"""The decoder-layer operators of this library on real work: cases, plain forms and exact values.

Three operators run next to the 4-bit GEMMs in every decoder layer of a served model:

* norm: root-mean-square norm of x + residual, written as fp16 / bf16, as int8 with one scale
  per row (what the W4A8 GEMM takes) or as E4M3 with one E8M0 scale per 32 values (what the MX
  GEMM takes);
* rope: rotary positions applied to the new tokens' queries and keys, keys and values written
  to their slots of a paged cache (fp16, bf16 or E4M3 with a scale per head);
* attn: attention of one new token per sequence over that paged cache.

With ``own`` false, ``run`` computes them with elementary torch operations in 32 bits, rounded
once at the end; with ``own`` true it makes the library's calls.  ``exact`` states the same
definitions in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}
E4M3_MAX = 448.0
BYTES = {"fp16": 2, "bf16": 2, "e4m3": 1}


def _norm(m, h, dtype, out, residual, name=None):
    c = {"op": "norm", "m": m, "h": h, "dtype": dtype, "out": out, "residual": residual}
    return dict(c, name=name) if name else c


def _rope(t, q_heads, kv_heads, d, rot, interleaved, dtype, kv, page, context, scaled, name=None):
    c = {"op": "rope", "t": t, "q_heads": q_heads, "kv_heads": kv_heads, "d": d, "rot": rot,
         "interleaved": interleaved, "dtype": dtype, "kv": kv, "page": page, "context": context,
         "scaled": scaled}
    return dict(c, name=name) if name else c


def _attn(b, length, ragged, empty, q_heads, kv_heads, d, dtype, kv, page, window, lse, name=None):
    c = {"op": "attn", "b": b, "length": length, "ragged": ragged, "empty": empty,
         "q_heads": q_heads, "kv_heads": kv_heads, "d": d, "dtype": dtype, "kv": kv, "page": page,
         "window": window, "lse": lse}
    return dict(c, name=name) if name else c


def listed():
    return [
        # one token of a single stream through an 8192-wide layer: latency is all there is
        _norm(1, 8192, "bf16", "same", True, "norm_decode_m1"),
        # a small decode batch in front of the W4A8 GEMM: int8 rows and their scales
        _norm(8, 8192, "bf16", "i8", True, "norm_i8_m8"),
        # an odd batch in front of the MX GEMM, no residual (the first layer of a stack)
        _norm(13, 4096, "fp16", "mx", False, "norm_mx_m13"),
        # a 4096-token prompt through an 8192-wide layer: bandwidth is all there is
        _norm(4096, 8192, "bf16", "same", True, "norm_prefill_m4096"),
        # one new token: its 64 queries and 8 keys rotated, key and value appended
        _rope(1, 64, 8, 128, 128, False, "bf16", "bf16", 64, 8192, False, "rope_decode_t1"),
        # a 4096-token prompt of the same layer
        _rope(4096, 64, 8, 128, 128, False, "bf16", "bf16", 64, 4096, False, "rope_prefill_t4096"),
        # an odd chunk of a long prompt: interleaved pairs, half of each head rotated, positions
        # scaled past the trained range, 8-bit cache in small pages
        _rope(1003, 32, 32, 128, 64, True, "fp16", "e4m3", 16, 65536, True, "rope_part_e4m3_t1003"),
        # a single short conversation: few bytes, latency counts
        _attn(1, 777, False, False, 64, 8, 128, "bf16", "bf16", 64, 0, False, "attn_b1_l777"),
        # a ragged batch with a key-value head for each query head and some idle slots
        _attn(16, 4096, True, True, 32, 32, 128, "fp16", "fp16", 16, 0, True, "attn_heads32_b16"),
        # one very long document: the work must be split along the cache
        _attn(1, 131072, False, False, 64, 8, 128, "bf16", "bf16", 64, 0, False, "attn_b1_l131072"),
        # a full serving batch, lengths from a tenth of the longest to the longest
        _attn(64, 16384, True, False, 64, 8, 128, "bf16", "bf16", 64, 0, False, "attn_b64_l16384"),
        # 8-bit cache, narrow heads, a sliding window over longer sequences
        _attn(33, 9000, True, True, 32, 4, 64, "bf16", "e4m3", 32, 4096, False, "attn_e4m3_window"),
    ]


def _log(rng, lo, hi):
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return n if n != 3072 else n + 1


def draw(rng):
    op = rng.choice(["norm", "rope", "attn", "attn"])
    dtype = rng.choice(["fp16", "bf16"])
    if op == "norm":
        out = rng.choice(["same", "same", "i8", "mx"])
        if out == "same":  # any width, multiples of 8 most often
            h = _log(rng, 256, 16384)
            h = h if rng.random() < 0.3 else h // 8 * 8
        else:
            h = max(1, _log(rng, 256, 16384) // 128) * 128
        h = h if h != 3072 else 3200
        m = _log(rng, 1, min(8192, 4096 * 8192 // h))
        return _norm(m, h, dtype, out, rng.random() < 0.7)
    d = rng.choice([64, 64, 80, 96, 128, 128, 128, 256])
    kv = rng.choice([dtype, dtype, "e4m3"])
    kv_heads = rng.choice([1, 2, 4, 8, 8, 16, 32])
    q_heads = kv_heads * rng.choice([n for n in (1, 2, 3, 4, 7, 8, 12, 16) if n * kv_heads <= 96])
    page = rng.choice([8, 16, 16, 32, 64, 128])
    if op == "rope":
        rot = rng.choice([d, d, d // 2])
        most = max(1, 4096 * 80 * 128 // ((q_heads + 2 * kv_heads) * d))
        return _rope(_log(rng, 1, min(8192, most)), q_heads, kv_heads, d, rot, rng.random() < 0.5,
                     dtype, kv, page, 1 << rng.randint(13, 17), rng.random() < 0.5)
    b = _log(rng, 1, 64)
    most = 64 * 16384 * 8 * 128 // 2 // (b * kv_heads * d)
    return _attn(b, _log(rng, 1, max(2, min(131072, most))), rng.random() < 0.7,
                 rng.random() < 0.3, q_heads, kv_heads, d, dtype, kv, page,
                 rng.choice([0, 0, 0, _log(rng, 16, 8192)]), rng.random() < 0.3)


def _lengths(case):
    """The sequences' lengths, up to their order: all alike, or spread from a tenth of the longest
    to the longest (the golden ratio's multiples); one in five 0 where idle slots are asked for."""
    n, longest = case["b"], case["length"]
    got = []
    for i in range(n):
        share = 0.1 + 0.9 * ((1.0 - i * 0.6180339887498949) % 1.0) if case["ragged"] and i else 1.0
        got.append(0 if case["empty"] and i % 5 == 4 else max(1, int(longest * share)))
    return got


def _read(case, length):
    """Cached tokens that one sequence's new token attends to."""
    return min(length, case["window"]) if case["window"] else length


def work(case):
    e = 2
    if case["op"] == "norm":
        m, h = case["m"], case["h"]
        out = {"same": e * m * h, "i8": m * h + 4 * m, "mx": m * h + m * h // 32}[case["out"]]
        moved = e * m * h * (3 if case["residual"] else 1) + e * h + out
        return {"bytes": moved, "flops": (5 if case["residual"] else 4) * m * h}
    d, hq, hkv = case["d"], case["q_heads"], case["kv_heads"]
    if case["op"] == "rope":
        t = case["t"]
        moved = t * (e * d * (2 * hq + 2 * hkv) + 2 * BYTES[case["kv"]] * hkv * d + 4 * case["rot"] + 12)
        return {"bytes": moved, "flops": 3 * t * (hq + hkv) * case["rot"]}
    read = sum(_read(case, n) for n in _lengths(case))
    moved = (read * 2 * hkv * d * BYTES[case["kv"]] + 2 * e * case["b"] * hq * d
             + 4 * case["b"] + 4 * sum(-(-_read(case, n) // case["page"]) for n in _lengths(case))
             + (4 * case["b"] * hq if case["lse"] else 0))
    return {"bytes": moved, "flops": 4 * read * hq * d}


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(shape, dtype, g, scale=1.0):
    wide = torch.float16 if dtype == torch.float8_e4m3fn else dtype
    x = torch.randn(shape, generator=g, device="cuda", dtype=wide).mul_(scale)
    return x.to(dtype)


def _pages(count, page, heads, d, kv, g):
    """A cache's key or value pages as a model leaves them: unit normal values (8-bit caches hold
    them over the head's scale)."""
    return _normal((count, page, heads, d), DTYPES[kv], g, 16.0 if kv == "e4m3" else 1.0)


def prepare(case, seed):
    g = _gen(seed)
    dtype = DTYPES[case["dtype"]]
    s = {"case": case}
    if case["op"] == "norm":
        m, h = case["m"], case["h"]
        s["x"] = _normal((m, h), dtype, g)
        # a residual stream with a few strong channels, as trained models have
        s["residual"] = None
        if case["residual"]:
            strong = torch.rand(h, generator=g, device="cuda") < 0.002
            s["residual"] = (_normal((m, h), torch.float32, g, 2.0) * (1.0 + 7.0 * strong)).to(dtype)
        s["weight"] = (1.0 + 0.1 * torch.randn(h, generator=g, device="cuda")).to(dtype)
        s["eps"] = 1e-5
        s["residual_out"] = torch.empty_like(s["x"]) if case["residual"] else None
        if case["out"] == "same":
            s["y"] = torch.empty_like(s["x"])
        elif case["out"] == "i8":
            s["codes"] = torch.empty((m, h), dtype=torch.int8, device="cuda")
            s["scale"] = torch.empty(m, dtype=torch.float32, device="cuda")
            s["y"] = torch.empty_like(s["x"])
        else:
            s["codes"] = torch.empty((m, h), dtype=torch.uint8, device="cuda")
            s["scale"] = torch.empty((m, h // 32), dtype=torch.uint8, device="cuda")
    elif case["op"] == "rope":
        t, d, hq, hkv, page = case["t"], case["d"], case["q_heads"], case["kv_heads"], case["page"]
        s["qkv"] = _normal((t, (hq + 2 * hkv) * d), dtype, g)  # one fused projection's output
        # rotation table: cos and sin of position x frequency, [position][rot]
        j = torch.arange(case["rot"] // 2, device="cuda", dtype=torch.float64)
        freq = 10000.0 ** (-2.0 * j / case["rot"]) / (4.0 if case["scaled"] else 1.0)
        angle = torch.arange(case["context"], device="cuda", dtype=torch.float64)[:, None] * freq
        s["table"] = torch.cat([angle.cos(), angle.sin()], 1).float()
        # one sequence's chunk when it is long, a batch of unrelated tokens when it is short
        if t > 64:
            first = int(torch.randint(0, max(1, case["context"] - t), (1,), generator=g, device="cuda"))
            s["positions"] = (first + torch.arange(t, device="cuda")).clamp_(max=case["context"] - 1).int()
        else:
            s["positions"] = torch.randint(0, case["context"], (t,), generator=g, device="cuda").int()
        count = -(-t // page) + 4
        order = torch.randperm(count, generator=g, device="cuda")
        i = torch.arange(t, device="cuda")
        s["slots"] = order[i // page] * page + i % page
        s["k"], s["v"] = (_pages(count, page, hkv, d, case["kv"], g) for _ in range(2))
        s["q_out"] = torch.empty((t, hq * d), dtype=dtype, device="cuda")
    else:
        b, d, hq, hkv, page = case["b"], case["d"], case["q_heads"], case["kv_heads"], case["page"]
        lengths = torch.tensor(_lengths(case), device="cuda")[torch.randperm(b, generator=g, device="cuda")]
        columns = -(-case["length"] // page)
        count = b * columns + 1
        s["q"] = _normal((b, hq * d), dtype, g, 1.5)
        s["k"], s["v"] = (_pages(count, page, hkv, d, case["kv"], g) for _ in range(2))
        s["pages"] = torch.randperm(count, generator=g, device="cuda")[: b * columns].view(b, columns).int()
        s["lengths"] = lengths.int()
        # what lies in a page past a sequence's end is left from another one: any bits
        last = lengths % page
        at = (s["pages"].long().gather(1, (lengths // page).clamp(max=columns - 1)[:, None]).squeeze(1))
        raw = 0x7F if case["kv"] == "e4m3" else 0x7FFF
        stale = ((torch.arange(page, device="cuda") >= last[:, None]) & (lengths % page != 0)[:, None])
        for x in (s["k"], s["v"]):
            bits = x.view(torch.uint8 if case["kv"] == "e4m3" else torch.int16)
            bits[at] = bits[at].masked_fill(stale[:, :, None, None], raw)
        s["out"] = torch.empty((b, hq * d), dtype=dtype, device="cuda")
        s["lse"] = torch.empty((b, hq), dtype=torch.float32, device="cuda") if case["lse"] else None
    if case["op"] != "norm":
        # 8-bit caches: the value of a stored number is the number times its head's scale
        s["k_scale"], s["v_scale"] = ((0.05 + 0.02 * torch.rand(case["kv_heads"], generator=g, device="cuda"))
                                      if case["kv"] == "e4m3" else None for _ in range(2))
    if own:  # the handles that a serving program keeps: cache, rotation, launch settings, workspace
        import weight_only_int4_tma_gb300 as w4
        s["w4"] = w4
        s["code"] = w4.W4A16_FP16 if case["dtype"] == "fp16" else w4.W4A16_BF16
        if case["op"] != "norm":
            s["cache"] = w4.kv_cache(s["k"], s["v"], s["k_scale"], s["v_scale"])
        if case["op"] == "rope":
            s["plan"] = w4.rope_config(hq, hkv, d, s["code"], s["table"], case["rot"],
                                       w4.DEC_ROPE_INTERLEAVED if case["interleaved"] else w4.DEC_ROPE_HALF,
                                       ldq=s["qkv"].stride(0), ldk=s["qkv"].stride(0), ldv=s["qkv"].stride(0))
            s["parts"] = [s["qkv"][:, : hq * d], s["qkv"][:, hq * d: (hq + hkv) * d], s["qkv"][:, (hq + hkv) * d:]]
        elif case["op"] == "attn":
            s["plan"] = w4.attn_config(hq, s["code"], d ** -0.5, s["pages"].shape[1], window=case["window"])
            s["workspace"] = w4.attn_workspace(s["plan"], s["cache"])
    return s


def run(state):
    return {"norm": _run_norm, "rope": _run_rope, "attn": _run_attn}[state["case"]["op"]](state)


def _run_norm(s):
    c = s["case"]
    if own:
        w4 = s["w4"]
        args = (s["x"], s["residual"], s["weight"], c["m"], c["h"], s["code"], s["eps"], s["residual_out"])
        if c["out"] == "same":
            w4.dec_rms_norm(*args, s["y"])
            return {"y": s["y"], "residual": s["residual_out"]}
        if c["out"] == "i8":
            w4.dec_rms_norm_i8(*args, s["codes"], s["scale"])
            torch.mul(s["codes"], s["scale"][:, None], out=s["y"])
            return {"y": s["y"], "scale": s["scale"], "residual": s["residual_out"]}
        w4.dec_rms_norm_mx(*args, s["codes"], s["scale"])
        return {"y": s["codes"].view(torch.float8_e4m3fn), "scale": s["scale"].view(torch.float8_e8m0fnu),
                "residual": s["residual_out"]}
    dtype = s["x"].dtype
    h = s["x"].float()
    if c["residual"]:
        h = h + s["residual"].float()
    y = h * torch.rsqrt(h.square().mean(1, keepdim=True) + s["eps"]) * s["weight"].float()
    residual = h.to(dtype) if c["residual"] else None
    if c["out"] == "same":
        return {"y": y.to(dtype), "residual": residual}
    if c["out"] == "i8":
        most = y.abs().amax(1)
        scale = torch.where(most > 0, most / 127.0, torch.ones_like(most))
        codes = torch.round(y / scale[:, None]).clamp(-127, 127)
        return {"y": (codes * scale[:, None]).to(dtype), "scale": scale, "residual": residual}
    blocks = y.view(c["m"], -1, 32)
    # the largest power of two in each block, by the exponent that frexp gives
    exponent = torch.frexp(blocks.abs().amax(2)).exponent - 1 - 8
    exponent = torch.where(blocks.abs().amax(2) > 0, exponent, -127).clamp(-127, 127)
    codes = torch.ldexp(blocks, -exponent[:, :, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return {"y": codes.view(c["m"], c["h"]), "scale": (exponent + 127).to(torch.uint8).view(torch.float8_e8m0fnu),
            "residual": residual}


def _turn(x, cos, sin, rot, interleaved):
    """The first `rot` values of each head of x [t, heads, d], turned by the tokens' angles."""
    head = x[..., :rot]
    if interleaved:
        a, b = head[..., 0::2], head[..., 1::2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = head[..., : rot // 2], head[..., rot // 2:]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([turned, x[..., rot:]], -1)


def _run_rope(s):
    c = s["case"]
    if own:
        s["w4"].dec_rope_append(s["plan"], s["cache"], *s["parts"], c["t"], s["positions"], s["slots"], s["q_out"])
        return {"q": s["q_out"], "k": s["k"], "v": s["v"]}
    t, d, hq, hkv = c["t"], c["d"], c["q_heads"], c["kv_heads"]
    x = s["qkv"].float().view(t, hq + 2 * hkv, d)
    row = s["table"][s["positions"].long()]
    cos, sin = row[:, None, : c["rot"] // 2], row[:, None, c["rot"] // 2:]
    turned = _turn(x[:, : hq + hkv], cos, sin, c["rot"], c["interleaved"])
    q, k, v = turned[:, :hq], turned[:, hq:], x[:, hq + hkv:]
    if c["kv"] == "e4m3":
        k = (k / s["k_scale"][:, None]).clamp(-E4M3_MAX, E4M3_MAX)
        v = (v / s["v_scale"][:, None]).clamp(-E4M3_MAX, E4M3_MAX)
    kind = torch.uint8 if c["kv"] == "e4m3" else s["k"].dtype
    s["k"].view(kind).view(-1, hkv, d)[s["slots"]] = k.to(s["k"].dtype).view(kind)
    s["v"].view(kind).view(-1, hkv, d)[s["slots"]] = v.to(s["v"].dtype).view(kind)
    return {"q": q.reshape(t, hq * d).to(s["qkv"].dtype), "k": s["k"], "v": s["v"]}


def _run_attn(s):
    c = s["case"]
    if own:
        s["w4"].dec_attn_paged(s["plan"], s["cache"], s["q"], s["pages"], s["lengths"], c["b"], s["out"],
                               s["lse"], s["workspace"])
        return {"out": s["out"], "lse": s["lse"]}
    b, d, hq, hkv = c["b"], c["d"], c["q_heads"], c["kv_heads"]
    kind = torch.uint8 if c["kv"] == "e4m3" else s["k"].dtype
    pages = s["pages"].long()

    def cached(x, scale):  # [b, kv heads, tokens, d] in 32 bits
        x = x.view(kind)[pages].view(x.dtype).flatten(1, 2).transpose(1, 2).float()
        return x if scale is None else x * scale[:, None, None]

    k, v = cached(s["k"], s["k_scale"]), cached(s["v"], s["v_scale"])
    at = torch.arange(k.shape[2], device=k.device)
    length = s["lengths"].long()[:, None]
    seen = at < length
    if c["window"]:
        seen = seen & (at >= length - c["window"])
    seen = seen[:, None, None, :]
    q = s["q"].float().view(b, hkv, hq // hkv, d)
    score = torch.matmul(q, k.transpose(2, 3)) * d ** -0.5
    score = score.masked_fill(~seen, -math.inf)
    most = score.amax(3, keepdim=True)
    p = torch.exp(score - most.masked_fill(most == -math.inf, 0.0))
    total = p.sum(3, keepdim=True)
    v = v.masked_fill(~seen.squeeze(2)[..., None], 0.0)
    out = torch.matmul(p, v) / total.masked_fill(total == 0, 1.0)
    lse = (most + total.log()).view(b, hq) if c["lse"] else None
    return {"out": out.view(b, hq * d).to(s["q"].dtype), "lse": lse}


def exact(case, seed):
    """What run() returns, from the operators' definitions in 64 bits."""
    s = prepare(case, seed)
    f64 = torch.float64
    if case["op"] == "norm":
        h = s["x"].to(f64) if s["residual"] is None else s["x"].to(f64) + s["residual"].to(f64)
        r = 1.0 / torch.sqrt((h * h).sum(1) / case["h"] + s["eps"])
        y = h * r[:, None] * s["weight"].to(f64)
        residual = h if case["residual"] else None
        if case["out"] == "same":
            return {"y": y, "residual": residual}
        if case["out"] == "i8":
            scale = y.abs().max(1).values / 127
            scale[scale == 0] = 1.0
            codes = torch.round(y / scale[:, None])
            return {"y": codes * scale[:, None], "scale": scale, "residual": residual}
        largest = y.view(case["m"], -1, 32).abs().max(2).values
        step = torch.floor(torch.log2(largest)).clamp(-119, 135) - 8
        scale = torch.exp2(step)
        z = (y.view(case["m"], -1, 32) / scale[:, :, None]).clamp(-448, 448)
        # E4M3 in 64 bits: three bits after the leading one, steps of 2^-9 below 2^-6
        unit = torch.exp2(torch.floor(torch.log2(z.abs().clamp_min(2.0 ** -6))) - 3)
        return {"y": (torch.round(z / unit) * unit).view(case["m"], case["h"]), "scale": scale, "residual": residual}
    d, hq, hkv = case["d"], case["q_heads"], case["kv_heads"]
    if case["op"] == "rope":
        if case["kv"] == "e4m3" and case["t"] * hkv * d > 1 << 27:
            return None
        t, half = case["t"], case["rot"] // 2
        x = s["qkv"].to(f64).view(t, hq + 2 * hkv, d)
        row = s["table"].to(f64)[s["positions"].long()]
        z = torch.complex(row[:, :half], row[:, half:])[:, None, :]
        turned = x[:, : hq + hkv].clone()
        first, second = ((slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if case["interleaved"]
                         else (slice(0, half), slice(half, 2 * half)))
        w = torch.complex(turned[..., first].contiguous(), turned[..., second].contiguous()) * z
        turned[..., first], turned[..., second] = w.real, w.imag
        cached = []
        for name, new in (("k", turned[:, hq:]), ("v", x[:, hq + hkv:])):
            pages = s[name].to(f64)
            if case["kv"] == "e4m3":
                new = (new / s[name + "_scale"].to(f64)[:, None]).clamp(-448, 448)
                unit = torch.exp2(torch.floor(torch.log2(new.abs().clamp_min(2.0 ** -6))) - 3)
                new = torch.round(new / unit) * unit
            pages.view(-1, hkv, d)[s["slots"]] = new
            cached.append(pages)
        return {"q": turned[:, :hq].reshape(t, hq * d), "k": cached[0], "v": cached[1]}
    out = torch.zeros((case["b"], hq, d), dtype=f64, device="cuda")
    lse = torch.full((case["b"], hq), -math.inf, dtype=f64, device="cuda")
    q = s["q"].to(f64).view(case["b"], hq, d)
    kind = torch.uint8 if case["kv"] == "e4m3" else s["k"].dtype
    for i, n in enumerate(s["lengths"].tolist()):
        n0 = max(0, n - case["window"]) if case["window"] else 0
        if n <= n0:
            continue
        tokens = torch.arange(n0, n, device="cuda")
        page, slot = s["pages"][i].long()[tokens // case["page"]], tokens % case["page"]
        for g in range(hkv):
            heads = slice(g * (hq // hkv), (g + 1) * (hq // hkv))
            kg, vg = (x.view(kind)[page, slot, g].view(x.dtype).to(f64) for x in (s["k"], s["v"]))
            if case["kv"] == "e4m3":
                kg, vg = kg * s["k_scale"][g].to(f64), vg * s["v_scale"][g].to(f64)
            score = q[i, heads] @ kg.T / math.sqrt(d)
            out[i, heads] = torch.softmax(score, 1) @ vg
            lse[i, heads] = torch.logsumexp(score, 1)
    return {"out": out.view(case["b"], hq * d), "lse": lse if case["lse"] else None}
