"""One decoder layer of a served model, from this library's kernels alone.

    python examples/decoder_layer.py [--w4a8] [--batch B] [--prompt T] [--new N]

The layer is norm -> QKV projection -> rotary positions + cache append -> attention over the paged
cache -> output projection -> residual + norm -> feed-forward, with 4-bit weights everywhere.
With --w4a8 the first norm writes int8 rows and the QKV projection is the W4A8 GEMM.  A prompt
is written to the cache token by token (each token attends to all before it), then N tokens are
decoded; the script prints the time of a decode step and of the same step as a CUDA graph.

Weights are random: the point is how the calls fit together.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import weight_only_int4_tma_gb300 as w4  # noqa: E402

DTYPES = {torch.float16: w4.W4A16_FP16, torch.bfloat16: w4.W4A16_BF16}
GROUP = 128


def random_w4a16(n, k, dtype, gen):
    """A packed W4A16 weight of n x k: symmetric codes, scales that keep outputs near unit size."""
    codes = torch.randint(-(1 << 31), 1 << 31, (n, k // 8), generator=gen, device="cuda",
                          dtype=torch.int64).to(torch.int32)
    scales = (torch.rand(k // GROUP, n, generator=gen, device="cuda") * 0.5 + 0.75) * 0.22 * k ** -0.5
    return w4.repack(codes, scales.to(dtype), None, n, k, GROUP, DTYPES[dtype])


def random_w4a8(n, k, gen):
    """A packed W4A8 weight: step 8 and offset 68 spread the codes over -60 .. 60."""
    codes = torch.randint(-(1 << 31), 1 << 31, (n, k // 8), generator=gen, device="cuda",
                          dtype=torch.int64).to(torch.int32)
    step = torch.full((n, k // GROUP), 8, dtype=torch.uint8, device="cuda")
    offset = torch.full((n, k // GROUP), 68, dtype=torch.uint8, device="cuda")
    scale = torch.full((n,), 0.028 * k ** -0.5, device="cuda")
    packed = torch.empty(w4.w4a8_packed_bytes(n, k), dtype=torch.uint8, device="cuda")
    w4.w4a8_repack(codes, step, offset, scale, n, k, packed)
    return packed


class DecoderLayer:
    """Weights, cache and buffers of one layer for a fixed batch of sequences."""

    def __init__(self, batch, hidden, q_heads, kv_heads, head_dim, ffn, max_len, *,
                 dtype=torch.bfloat16, kv_dtype=None, page_size=16, w4a8=False, rot_dim=None, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.B, self.H, self.F, self.dtype, self.code, self.w4a8 = batch, hidden, ffn, dtype, DTYPES[dtype], w4a8
        self.hq, self.hkv, self.D, self.page = q_heads, kv_heads, head_dim, page_size
        self.nq, self.nkv = q_heads * head_dim, kv_heads * head_dim
        nqkv = self.nq + 2 * self.nkv
        self.norm1, self.norm2 = ((1 + 0.1 * torch.randn(hidden, generator=g, device="cuda")).to(dtype)
                                  for _ in range(2))
        self.wqkv = random_w4a8(nqkv, hidden, g) if w4a8 else random_w4a16(nqkv, hidden, dtype, g)
        self.wo = random_w4a16(hidden, self.nq, dtype, g)
        self.w1, self.w2 = random_w4a16(ffn, hidden, dtype, g), random_w4a16(hidden, ffn, dtype, g)

        # the paged cache, its block table (here: pages dealt out at random) and lengths
        columns = -(-max_len // page_size)
        kv_dtype = kv_dtype or dtype
        shape = (batch * columns, page_size, kv_heads, head_dim)
        self.k, self.v = (torch.zeros(shape, dtype=dtype, device="cuda").to(kv_dtype) for _ in range(2))
        self.kv_scale = torch.full((kv_heads,), 0.03, device="cuda") if kv_dtype == torch.float8_e4m3fn else None
        self.cache = w4.kv_cache(self.k, self.v, self.kv_scale, self.kv_scale)
        self.pages = torch.randperm(batch * columns, generator=g, device="cuda").view(batch, columns).int()
        self.lens = torch.zeros(batch, dtype=torch.int32, device="cuda")

        rot_dim = rot_dim or head_dim
        self.table = torch.empty(max_len, rot_dim, device="cuda")
        w4.dec_rope_table(rot_dim, 10000.0, None, self.table, max_len)
        self.rope = w4.rope_config(q_heads, kv_heads, head_dim, self.code, self.table, rot_dim,
                                   ldq=nqkv, ldk=nqkv, ldv=nqkv)
        self.attn = w4.attn_config(q_heads, self.code, head_dim ** -0.5, columns)
        self.workspace = w4.attn_workspace(self.attn, self.cache)

        def buf(n):
            return torch.empty(batch, n, dtype=dtype, device="cuda")
        self.y, self.qkv, self.q, self.a, self.o, self.h, self.u = (
            buf(n) for n in (hidden, nqkv, self.nq, self.nq, hidden, hidden, ffn))
        self.y_i8 = torch.empty(batch, hidden, dtype=torch.int8, device="cuda")
        self.s_y = torch.empty(batch, device="cuda")
        self.positions = torch.empty(batch, dtype=torch.int32, device="cuda")
        self.slots = torch.empty(batch, dtype=torch.int64, device="cuda")

    def advance(self):
        """One more token per sequence: its position, its slot in the cache, the new lengths."""
        self.positions.copy_(self.lens)
        page = self.pages.gather(1, (self.lens // self.page).long()[:, None]).squeeze(1)
        self.slots.copy_(page.long() * self.page + self.lens % self.page)
        self.lens += 1

    def step(self, x, out):
        """out = the layer's output for one token per sequence, x [B, H]; library calls only."""
        B, H, code, eps = self.B, self.H, self.code, 1e-5
        nqkv, nq, nkv = self.qkv.shape[1], self.nq, self.nkv
        if self.w4a8:
            w4.dec_rms_norm_i8(x, None, self.norm1, B, H, code, eps, None, self.y_i8, self.s_y)
            w4.w4a8_gemm(self.y_i8, self.s_y, self.wqkv, B, nqkv, H, code, self.qkv)
        else:
            w4.dec_rms_norm(x, None, self.norm1, B, H, code, eps, None, self.y)
            w4.w4a16_gemm(self.y, self.wqkv, B, nqkv, H, GROUP, code, self.qkv)
        w4.dec_rope_append(self.rope, self.cache, self.qkv, self.qkv[:, nq:nq + nkv], self.qkv[:, nq + nkv:], B,
                           self.positions, self.slots, self.q)
        w4.dec_attn_paged(self.attn, self.cache, self.q, self.pages, self.lens, B, self.a, None, self.workspace)
        w4.w4a16_gemm(self.a, self.wo, B, H, nq, GROUP, code, self.o)
        w4.dec_rms_norm(self.o, x, self.norm2, B, H, code, eps, self.h, self.y)
        w4.w4a16_gemm_epilogue(self.y, self.w1, B, self.F, H, GROUP, code, None, None, w4.W4A16_ACT_SILU, self.u)
        w4.w4a16_gemm_epilogue(self.u, self.w2, B, H, self.F, GROUP, code, None, self.h, w4.W4A16_ACT_NONE, out)


def _time(f, n):
    a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    a.record()
    for _ in range(n):
        f()
    b.record()
    torch.cuda.synchronize()
    return a.elapsed_time(b) / n * 1e3


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--w4a8", action="store_true")
    ap.add_argument("--kv8", action="store_true", help="8-bit (E4M3) cache")
    ap.add_argument("--batch", type=int, default=8)
    ap.add_argument("--prompt", type=int, default=1000)
    ap.add_argument("--new", type=int, default=32)
    a = ap.parse_args()
    layer = DecoderLayer(a.batch, 8192, 64, 8, 128, 28672, a.prompt + a.new + 64, page_size=64, w4a8=a.w4a8,
                         kv_dtype=torch.float8_e4m3fn if a.kv8 else None)
    x = torch.randn(a.batch, 8192, device="cuda").to(torch.bfloat16)
    out = torch.empty_like(x)
    for _ in range(a.prompt + a.new):
        layer.advance()
        layer.step(x, out)
        x.copy_(out / out.float().square().mean(1, keepdim=True).sqrt().to(out.dtype))
    layer.advance()
    layer.step(x, out)
    eager = _time(lambda: layer.step(x, out), 100)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer.step(x, out)
    replay = _time(graph.replay, 100)
    st = w4.w4a16_get_device_status()
    assert st == 0, w4.status_string(st)
    print(f"batch {a.batch}, {int(layer.lens[0])} tokens each: {eager:.1f} us a step, {replay:.1f} us as a graph")


if __name__ == "__main__":
    main()
