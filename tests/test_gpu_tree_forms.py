"""Attention of drafted trees: large row counts over long contexts, and batches with a sequence that is refused."""
import pytest
import torch

import weight_only_int4_tma_gb300 as w4

from test_gpu_tree import MARK, Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,kv,d", [("bf16", "bf16", 128), ("fp16", "fp16", 64), ("bf16", "e4m3", 128), ("bf16", "bf16", 256)])
def test_many_rows_over_long_contexts(dtype, kv, d):
    """512 rows of a head over more than 5000 tokens, cut into parts; fewer beside them."""
    Case([(9000, 64), (5301, 33), (700, 1)], 8, 1, d, dtype, kv, page=64, seed=50 + d).run().check()


@pytest.mark.parametrize("what", ["long", "negative", "short", "beyond", "too_many", "descending", "before"])
def test_the_other_sequences_of_a_bad_batch(what):
    """A sequence out of range is left out, its rows as they were; all others are right."""
    c = Case([(90, 8), (60, 12), (100, 5)], 4, 2, 64, "bf16", seed=51, pad=(0, 70))
    args = c.args()
    good = [0, 2]
    if what == "long":
        c.lens[1] = c.pages.shape[1] * 16 + 1
    if what == "negative":
        c.lens[1] = -1
    if what == "short":
        c.lens[1] = 11
    if what == "beyond":            # nothing is left for the third
        c.dev_starts[2:], good = c.T + 1, [0]
    if what == "too_many":          # likewise
        c.dev_starts[2:], good = 8 + 65, [0]
    if what == "descending":        # likewise
        c.dev_starts[2:], good = 3, [0]
    if what == "before":
        c.dev_starts[0], good = -1, [1, 2]
    w4.dec_attn_tree(*args)
    assert w4.w4a16_get_device_status() == w4.W4A16_ERR_INVALID_ARG
    c.seqs = [(ctx, n if b in good else 0) for b, (ctx, n) in enumerate(c.seqs)]
    c.check()                       # rows of no good sequence hold the mark
    touched = sum(n for _, n in c.seqs)
    assert int((c.out == MARK).all(1).sum()) == c.T - touched
