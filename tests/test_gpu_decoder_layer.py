"""The example layer (examples/decoder_layer.py) against the same layer in 64 bits.

The library's layer rounds to the activation type after the norms, the projections, the rotation,
the attention and the feed-forward's two halves: nine roundings of at most U relative each (and
one of the weights' products and of the cached keys and values), so the outputs may differ by
12 U in the 2-norm; the int8 rows add 1/127 of the row's largest value over sqrt(3), the 8-bit
cache 2^-4 over sqrt(3) in the keys and values."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
F64 = torch.float64
U = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}


def _dequant(packed, n, k, dtype):
    import weight_only_int4_tma_gb300 as w4
    from decoder_layer import DTYPES, GROUP
    W = torch.empty(n, k, dtype=dtype, device="cuda")
    w4.w4a16_dequant_debug(packed, n, k, GROUP, DTYPES[dtype], W)
    return W.to(F64)


def _weights(layer):
    import weight_only_int4_tma_gb300 as w4
    nqkv = layer.qkv.shape[1]
    if layer.w4a8:
        W = torch.empty(nqkv, layer.H, dtype=torch.int8, device="cuda")
        w4.w4a8_dequant_debug(layer.wqkv, nqkv, layer.H, W)
        wqkv = W.to(F64) * (0.028 * layer.H ** -0.5)
    else:
        wqkv = _dequant(layer.wqkv, nqkv, layer.H, layer.dtype)
    return (wqkv, _dequant(layer.wo, layer.H, layer.nq, layer.dtype),
            _dequant(layer.w1, layer.F, layer.H, layer.dtype), _dequant(layer.w2, layer.H, layer.F, layer.dtype))


def _plain_step(layer, weights, x, position, keys, values):
    """One token of every sequence in 64 bits; keys and values grow by it."""
    from oracle import layer as ol
    wqkv, wo, w1, w2 = weights
    B, D = layer.B, layer.D
    _, y = ol.rms_norm(x, None, layer.norm1, 1e-5)
    qkv = y @ wqkv.T
    q, k, v = qkv[:, :layer.nq], qkv[:, layer.nq:layer.nq + layer.nkv], qkv[:, layer.nq + layer.nkv:]
    rows = layer.table[position].to(F64)[None].expand(B, -1)
    q, _ = ol.rope(q.reshape(B, layer.hq, D), rows, layer.table.shape[1], False)
    k, _ = ol.rope(k.reshape(B, layer.hkv, D), rows, layer.table.shape[1], False)
    keys.append(k)
    values.append(v.reshape(B, layer.hkv, D))
    K, V = torch.stack(keys, 1), torch.stack(values, 1)
    out = torch.empty(B, layer.hq, D, dtype=F64, device="cuda")
    G = layer.hq // layer.hkv
    for b in range(B):
        for h in range(layer.hq):
            out[b, h] = ol.attn(q[b, h], K[b, :, h // G], V[b, :, h // G], D ** -0.5)[0]
    h = x.to(F64) + out.reshape(B, -1) @ wo.T
    _, y = ol.rms_norm(h, None, layer.norm2, 1e-5)
    u = y @ w1.T
    return h + (u * torch.sigmoid(u)) @ w2.T


@pytest.mark.parametrize("dtype,w4a8,kv8", [(torch.bfloat16, False, False), (torch.float16, False, False),
                                            (torch.float16, True, False), (torch.bfloat16, False, True)], ids=str)
def test_layer_matches_64_bits(dtype, w4a8, kv8):
    import weight_only_int4_tma_gb300 as w4
    from decoder_layer import DecoderLayer
    B, steps = 3, 37
    layer = DecoderLayer(B, 512, 8, 2, 64, 1024, 64, dtype=dtype, w4a8=w4a8,
                         kv_dtype=torch.float8_e4m3fn if kv8 else None, seed=4)
    weights = _weights(layer)
    g = torch.Generator(device="cuda").manual_seed(9)
    keys, values, out = [], [], torch.empty(B, 512, dtype=dtype, device="cuda")
    tol = 12 * U[dtype] + (0.02 if w4a8 else 0) + (2.0 ** -4 / 3 ** 0.5 if kv8 else 0)
    for t in range(steps):
        x = torch.randn(B, 512, generator=g, device="cuda").to(dtype)
        layer.advance()
        layer.step(x, out)
        want = _plain_step(layer, weights, x, t, keys, values)
        rel = float(torch.linalg.norm(out.to(F64) - want) / torch.linalg.norm(want))
        assert rel <= tol, (t, rel, tol)
    assert w4.w4a16_get_device_status() == 0 and layer.lens.tolist() == [steps] * B


def test_layer_as_a_graph_gives_the_same_bits():
    from decoder_layer import DecoderLayer
    layer = DecoderLayer(4, 512, 8, 2, 64, 1024, 64, seed=1)
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn(4, 512, generator=g, device="cuda").to(torch.bfloat16)
    out = torch.empty_like(x)
    layer.advance()
    layer.step(x, out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer.step(x, out)
    for _ in range(20):
        x.copy_(torch.randn(4, 512, generator=g, device="cuda"))
        layer.advance()
        layer.step(x, out)
        want = out.clone()
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
