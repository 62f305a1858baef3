"""Refusals of the operators of drafted tokens (include/decode.h): every bad argument is answered on
the host, before anything is launched, so these need no GPU."""
import math

import pytest

import weight_only_int4_tma_gb300 as w4
from weight_only_int4_tma_gb300 import build as w4build

BAD, UNSUP, OK = w4.W4A16_ERR_INVALID_ARG, w4.W4A16_ERR_UNSUPPORTED, w4.W4A16_OK
F = 1 << 20  # an aligned address that is never dereferenced


@pytest.fixture(scope="module")
def L():
    w4build.build()
    return w4.lib()


def _cache(**change):
    c = w4.KvCache(F, F, None, None, 64 * 256, 256, 64, 64 * 256, 256, 64, 10, 64, 4, 64, 0, 0)
    for k, v in change.items():
        setattr(c, k, v)
    return c


CACHE_FAULTS = [(dict(k=None), BAD), (dict(v=F + 8), BAD), (dict(num_pages=0), BAD),
                (dict(page_size=0), BAD), (dict(reserved=1), BAD), (dict(dtype=3), UNSUP),
                (dict(k_slot_stride=-256), BAD), (dict(v_head_stride=68), BAD), (dict(k_scale=F + 2), BAD),
                (dict(head_dim=68), UNSUP), (dict(head_dim=264), UNSUP), (dict(dtype=2, head_dim=72), UNSUP)]


def tree(L, cfg=None, cache=None, **change):
    a = dict(q=F, table=F, lens=F, starts=F, mask=F, B=2, T=9, out=F, lse=F, ws=F, n=1 << 40)
    a.update(change)
    cfg = w4.TreeConfig(8, 0, 20, 0, 0, 0.125, 0, 0, 0) if cfg is None else cfg
    return L.dec_attn_tree(cfg, _cache() if cache is None else cache, *a.values(), None)


@pytest.mark.parametrize("change,want", CACHE_FAULTS + [
    (dict(kv_heads=3), BAD), (dict(dtype=1), UNSUP), (dict(page_size=1 << 30), UNSUP)], ids=str)
def test_tree_cache_refusals(L, change, want):
    assert tree(L, cache=_cache(**change)) == want
    assert L.dec_attn_tree_workspace_bytes(w4.TreeConfig(8, 0, 20, 0, 0, 0.125, 0, 0, 0), _cache(**change)) == 0


@pytest.mark.parametrize("change,want", [
    (dict(q_heads=0), BAD), (dict(q_heads=6), BAD), (dict(q_heads=(1 << 20) + 4), UNSUP), (dict(dtype=2), UNSUP),
    (dict(max_pages=0), BAD), (dict(window=-1), BAD), (dict(sinks=-1), BAD), (dict(scale=math.nan), BAD),
    (dict(scale=math.inf), BAD), (dict(ldq=504), BAD), (dict(ldo=516), UNSUP), (dict(ld_table=19), BAD),
    (dict(max_pages=1 << 26), UNSUP)], ids=str)
def test_tree_config_refusals(L, change, want):
    cfg = w4.TreeConfig(8, 0, 20, 0, 0, 0.125, 0, 0, 0)
    for k, v in change.items():
        setattr(cfg, k, v)
    assert tree(L, cfg) == want


def test_tree_argument_refusals(L):
    assert tree(L, B=0) == OK and tree(L, T=0) == OK and tree(L, B=-1) == BAD and tree(L, T=-1) == BAD
    assert tree(L, B=(1 << 24) + 1) == UNSUP
    for bad in (dict(q=None), dict(table=None), dict(lens=None), dict(starts=None), dict(out=None), dict(ws=None),
                dict(q=F + 8), dict(out=F + 2), dict(table=F + 2), dict(lens=F + 1), dict(starts=F + 2),
                dict(mask=F + 4), dict(lse=F + 2), dict(ws=F + 8)):
        assert tree(L, **bad) == BAD, bad
    assert L.dec_attn_tree(None, _cache(), F, F, F, F, F, 2, 9, F, F, F, 1 << 40, None) == BAD
    cfg = w4.TreeConfig(8, 0, 20, 0, 0, 0.125, 0, 0, 0)
    assert L.dec_attn_tree(cfg, None, F, F, F, F, F, 2, 9, F, F, F, 1 << 40, None) == BAD


@pytest.mark.parametrize("change,want", [
    (dict(vocab=0), BAD), (dict(vocab=(1 << 24) + 1), UNSUP), (dict(dtype=3), UNSUP), (dict(dtype=-1), UNSUP),
    (dict(n_ids=-1), BAD), (dict(n_ids=65537), UNSUP), (dict(top=-1), BAD), (dict(top=33), UNSUP),
    (dict(vocab=5, top=6), BAD), (dict(ld=99), BAD), (dict(ld=-1), BAD)], ids=str)
def test_logprob_config_refusals(L, change, want):
    cfg = w4.LogprobConfig(100, 0, 1, 5, 0)
    for k, v in change.items():
        setattr(cfg, k, v)
    assert L.dec_token_logprobs(cfg, F, F, F, 3, F, F, F, F, F, None) == want


def test_logprob_argument_refusals(L):
    cfg = w4.LogprobConfig(100, 2, 1, 5, 0)
    names = "x factor ids T lp lse ent tid tlp".split()

    def call(**change):
        a = dict(zip(names, (F, F, F, 3, F, F, F, F, F)))
        a.update(change)
        return L.dec_token_logprobs(cfg, *a.values(), None)
    assert call(T=0) == OK and call(T=-1) == BAD
    for bad in (dict(x=None), dict(ids=None), dict(lp=None), dict(tid=None), dict(x=F + 2), dict(factor=F + 1),
                dict(ids=F + 2), dict(lp=F + 1), dict(lse=F + 2), dict(ent=F + 2), dict(tid=F + 1), dict(tlp=F + 3)):
        assert call(**bad) == BAD, bad
    assert L.dec_token_logprobs(None, F, F, F, 3, F, F, F, F, F, None) == BAD


@pytest.mark.parametrize("change,want", CACHE_FAULTS + [(dict(kv_heads=(1 << 20) + 1), UNSUP)], ids=str)
def test_move_cache_refusals(L, change, want):
    assert L.dec_kv_move(_cache(**change), F, F, F, 2, 3, None) == want


@pytest.mark.parametrize("stride", ["k_page_stride", "v_page_stride", "k_slot_stride", "v_slot_stride", "k_head_stride",
                                    "v_head_stride"])
def test_move_of_places_that_share_memory(L, stride):
    """Refused where there are several pages, slots or heads; of one, the stride does not matter."""
    assert L.dec_kv_move(_cache(**{stride: 0}), F, F, F, 2, 0, None) == BAD
    one = {"page": "num_pages", "slot": "page_size", "head": "kv_heads"}[stride.split("_")[1]]
    assert L.dec_kv_move(_cache(**{stride: 0, one: 1}), F, F, F, 2, 0, None) == OK


def test_move_argument_refusals(L):
    call = lambda src=F, dst=F, starts=F, B=2, N=3: L.dec_kv_move(_cache(), src, dst, starts, B, N, None)  # noqa: E731
    assert call(B=0) == OK and call(N=0) == OK and call(B=-1) == BAD and call(N=-1) == BAD
    for bad in (dict(src=None), dict(dst=None), dict(starts=None), dict(src=F + 4), dict(dst=F + 4), dict(starts=F + 2)):
        assert call(**bad) == BAD, bad
    assert L.dec_kv_move(None, F, F, F, 2, 3, None) == BAD


def test_tree_mask():
    assert w4.tree_mask([]) == []
    assert w4.tree_mask([-1, 0, 0, 1, -1, 4]) == [1, 3, 5, 11, 16, 48]
    assert w4.tree_mask(range(-1, 63))[63] == -1          # all 64 bits, as a signed number
    for bad in ([0], [-1, 1], [-2], [-1, 0, 3], [-1] * 65):
        with pytest.raises(w4.W4A16Error):
            w4.tree_mask(bad)


def test_configs():
    c = w4.tree_config(8, 1, 0.5, 20, window=7, sinks=3, ldq=8, ldo=16, ld_table=30)
    assert (c.q_heads, c.dtype, c.max_pages, c.window, c.sinks, c.scale) == (8, 1, 20, 7, 3, 0.5)
    assert (c.ldq, c.ldo, c.ld_table) == (8, 16, 30)
    c = w4.logprob_config(100, 2, n_ids=4, top=5, ld=104)
    assert (c.vocab, c.dtype, c.n_ids, c.top, c.ld) == (100, 2, 4, 5, 104)
