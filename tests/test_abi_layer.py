"""Refusals of the decoder-layer operators (include/decode.h): every bad argument is answered on
the host, before anything is launched, so these need no GPU."""
import ctypes

import pytest

import weight_only_int4_tma_gb300 as w4
from weight_only_int4_tma_gb300 import build as w4build

BAD, UNSUP, OK = w4.W4A16_ERR_INVALID_ARG, w4.W4A16_ERR_UNSUPPORTED, w4.W4A16_OK
F = 1 << 20  # an aligned address that is never dereferenced


@pytest.fixture(scope="module")
def L():
    w4build.build()
    return w4.lib()


@pytest.mark.parametrize("change,want", [
    (dict(M=0), OK), (dict(M=-1), BAD), (dict(H=0), BAD), (dict(H=(1 << 20) + 1), UNSUP),
    (dict(dtype=2), UNSUP), (dict(eps=-1.0), BAD), (dict(eps=float("nan")), BAD),
    (dict(eps=float("inf")), BAD), (dict(x=None), BAD), (dict(y=None), BAD),
    (dict(ldx=63), BAD), (dict(ldr=63), BAD), (dict(ldy=63), BAD), (dict(x=F + 1), BAD),
    (dict(residual=F + 1), BAD), (dict(weight=F + 1), BAD), (dict(rout=F + 1), BAD),
    (dict(y=F + 1), BAD)], ids=str)
def test_norm_refusals(L, change, want):
    a = dict(x=F, ldx=0, residual=F, ldr=0, weight=F, M=2, H=64, dtype=0, eps=1e-5, rout=F, y=F, ldy=0)
    a.update(change)
    assert L.dec_rms_norm(*a.values(), None) == want


@pytest.mark.parametrize("change,want", [
    (dict(M=0), OK), (dict(H=68), UNSUP), (dict(H=32776), UNSUP), (dict(s=None), BAD),
    (dict(s=F + 2), BAD), (dict(y=F + 4), BAD), (dict(x=F + 8), BAD), (dict(ldx=68), BAD),
    (dict(ldr=68), BAD), (dict(weight=F + 2), BAD), (dict(rout=F + 2), BAD)], ids=str)
def test_norm_i8_refusals(L, change, want):
    a = dict(x=F, ldx=0, residual=F, ldr=0, weight=F, M=2, H=64, dtype=0, eps=1e-5, rout=F, y=F, s=F)
    a.update(change)
    assert L.dec_rms_norm_i8(*a.values(), None) == want


@pytest.mark.parametrize("change,want", [
    (dict(M=0), OK), (dict(H=72), UNSUP), (dict(H=32800), UNSUP), (dict(s=None), BAD),
    (dict(y=F + 4), BAD), (dict(residual=F + 2), BAD)], ids=str)
def test_norm_mx_refusals(L, change, want):
    a = dict(x=F, ldx=0, residual=F, ldr=0, weight=F, M=2, H=64, dtype=0, eps=1e-5, rout=F, y=F, s=F)
    a.update(change)
    assert L.dec_rms_norm_mx(*a.values(), None) == want


NAN = float("nan")


@pytest.mark.parametrize("rot,base,scaling,table,n,want", [
    (64, 1e4, None, F, 0, OK), (64, 1e4, None, None, 5, BAD), (64, 1e4, None, F + 4, 5, BAD),
    (64, 1.0, None, F, 5, BAD), (64, NAN, None, F, 5, BAD), (64, 1e4, None, F, -1, BAD),
    (63, 1e4, None, F, 5, UNSUP), (0, 1e4, None, F, 5, UNSUP), (258, 1e4, None, F, 5, UNSUP),
    (64, 1e4, (4, 1, 0, 1, 1, 0), F, 5, BAD), (64, 1e4, (1, 0, 0, 1, 1, 0), F, 5, BAD),
    (64, 1e4, (1, NAN, 0, 1, 1, 0), F, 5, BAD), (2, 1e4, (2, 4, 0, 1, 1, 0), F, 5, UNSUP),
    (64, 1e4, (3, 4, 2, 2, 1, 0), F, 5, BAD), (64, 1e4, (3, 4, 1, 2, 0, 0), F, 5, BAD),
    (64, 1e4, (0, 0, 0, 0, 0, -1.0), F, 5, BAD)], ids=str)
def test_rope_table_refusals(L, rot, base, scaling, table, n, want):
    s = w4.RopeScaling(*scaling) if scaling else None
    assert L.dec_rope_table(rot, base, s, table, n, None) == want


def _cache(**change):
    c = w4.KvCache(F, F, None, None, 64 * 256, 256, 64, 64 * 256, 256, 64, 10, 64, 4, 64, 0, 0)
    for k, v in change.items():
        setattr(c, k, v)
    return c


CACHE_FAULTS = [(dict(k=None), BAD), (dict(v=F + 8), BAD), (dict(num_pages=0), BAD),
                (dict(page_size=0), BAD), (dict(reserved=1), BAD), (dict(dtype=3), UNSUP),
                (dict(dtype=1), UNSUP), (dict(k_slot_stride=-256), BAD),
                (dict(v_head_stride=68), BAD), (dict(k_scale=F + 2), BAD)]


@pytest.mark.parametrize("change,want", CACHE_FAULTS + [(dict(kv_heads=5), BAD), (dict(head_dim=72), BAD)],
                         ids=str)
def test_rope_cache_refusals(L, change, want):
    cfg = w4.RopeConfig(8, 4, 64, 0, 64, 0, 100, 0, F, 0, 0, 0, 0, 0)
    assert L.dec_rope_append(cfg, _cache(**change), F, F, F, 3, F, F, F, None, None) == want


@pytest.mark.parametrize("change,want", [
    (dict(q_heads=-1), BAD), (dict(head_dim=0), BAD), (dict(head_dim=60), UNSUP),
    (dict(head_dim=264), UNSUP), (dict(dtype=2), UNSUP), (dict(rot_dim=63), UNSUP),
    (dict(rot_dim=66), BAD), (dict(rot_dim=-2), BAD), (dict(layout=2), BAD),
    (dict(table_len=-1), BAD), (dict(reserved=1), BAD), (dict(table=None), BAD),
    (dict(table=F + 4), BAD), (dict(ldq=504), BAD), (dict(ldk=260), UNSUP), (dict(ldqo=8), BAD)],
    ids=str)
def test_rope_config_refusals(L, change, want):
    cfg = w4.RopeConfig(8, 4, 64, 0, 64, 0, 100, 0, F, 0, 0, 0, 0, 0)
    for k, v in change.items():
        setattr(cfg, k, v)
    assert L.dec_rope_append(cfg, None, F, F, F, 3, F, F, F, None, None) == want


def test_rope_argument_refusals(L):
    cfg = w4.RopeConfig(8, 4, 64, 0, 64, 0, 100, 0, F, 0, 0, 0, 0, 0)
    call = lambda cache=_cache(), q=F, k=F, v=F, T=3, pos=F, slots=F, qo=F, ko=None: (  # noqa: E731
        L.dec_rope_append(cfg, cache, q, k, v, T, pos, slots, qo, ko, None))
    assert call(T=0) == OK and call(T=-1) == BAD
    for bad in (dict(q=None), dict(k=None), dict(v=None), dict(pos=None), dict(slots=None),
                dict(qo=None), dict(q=F + 8), dict(k=F + 2), dict(v=F + 2), dict(qo=F + 8),
                dict(ko=F + 8), dict(pos=F + 2), dict(slots=F + 4)):
        assert call(**bad) == BAD, bad
    assert L.dec_rope_append(None, None, F, F, F, 3, F, F, F, None, None) == BAD
    assert call(cache=_cache(dtype=2, head_dim=64, k_page_stride=8)) == BAD  # 8 bytes


@pytest.mark.parametrize("change,want", CACHE_FAULTS + [
    (dict(kv_heads=3), BAD), (dict(head_dim=68), UNSUP), (dict(head_dim=264), UNSUP),
    (dict(dtype=2, head_dim=72), UNSUP), (dict(page_size=1 << 30), UNSUP)], ids=str)
def test_attn_cache_refusals(L, change, want):
    cfg = w4.AttnConfig(8, 0, 20, 0, 0.125, 0, 0, 0, 0)
    assert L.dec_attn_paged(cfg, _cache(**change), F, F, F, 2, F, None, F, 1 << 40, None) == want
    assert L.dec_attn_workspace_bytes(cfg, _cache(**change)) == 0


@pytest.mark.parametrize("change,want", [
    (dict(q_heads=0), BAD), (dict(q_heads=6), BAD), (dict(dtype=2), UNSUP), (dict(dtype=1), UNSUP),
    (dict(max_pages=0), BAD), (dict(window=-1), BAD), (dict(scale=float("inf")), BAD),
    (dict(reserved=1), BAD), (dict(ldq=504), BAD), (dict(ldo=516), UNSUP), (dict(ld_table=19), BAD)],
    ids=str)
def test_attn_config_refusals(L, change, want):
    cfg = w4.AttnConfig(8, 0, 20, 0, 0.125, 0, 0, 0, 0)
    for k, v in change.items():
        setattr(cfg, k, v)
    assert L.dec_attn_paged(cfg, _cache(), F, F, F, 2, F, None, F, 1 << 40, None) == want


def test_attn_argument_refusals(L):
    cfg = w4.AttnConfig(8, 0, 20, 0, 0.125, 0, 0, 0, 0)
    call = lambda q=F, bt=F, lens=F, B=2, out=F, lse=None, ws=F: (  # noqa: E731
        L.dec_attn_paged(cfg, _cache(), q, bt, lens, B, out, lse, ws, 1 << 40, None))
    assert call(B=0) == OK and call(B=-1) == BAD
    for bad in (dict(q=None), dict(bt=None), dict(lens=None), dict(out=None), dict(ws=None),
                dict(q=F + 8), dict(bt=F + 2), dict(lens=F + 2), dict(out=F + 8), dict(lse=F + 2),
                dict(ws=F + 8)):
        assert call(**bad) == BAD, bad
    assert L.dec_attn_paged(None, _cache(), F, F, F, 2, F, None, F, 1 << 40, None) == BAD
    assert L.dec_attn_paged(cfg, None, F, F, F, 2, F, None, F, 1 << 40, None) == BAD


def test_structs_have_the_headers_sizes(tmp_path):
    """The binding's structs are laid out as the C compiler lays out the header's."""
    import os
    import subprocess
    src = tmp_path / "s.c"
    src.write_text('#include <stdio.h>\n#include "decode.h"\nint main(void) { printf("%zu %zu %zu %zu",'
                   " sizeof(dec_kv_cache), sizeof(dec_rope_scaling), sizeof(dec_rope_config),"
                   " sizeof(dec_attn_config)); return 0; }\n")
    exe = tmp_path / "s"
    subprocess.run(["gcc", "-I", os.path.dirname(w4.HEADER), str(src), "-o", str(exe)], check=True)
    got = [int(n) for n in subprocess.run([str(exe)], capture_output=True, text=True).stdout.split()]
    assert got == [ctypes.sizeof(t) for t in (w4.KvCache, w4.RopeScaling, w4.RopeConfig, w4.AttnConfig)]
