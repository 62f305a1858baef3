"""Attention of drafted tokens where its numbers come to an end: scales, weights that vanish, what is not finite."""
import pytest
import torch

from test_gpu_tree import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("window", [0, 50])
@pytest.mark.parametrize("scale,spread", [(2.0 ** -40, 2.0 ** -112), (2.0 ** -126, 2.0 ** -60), (2.0 ** -20, 2.0 ** -114),
                                          (1e-44, 1.0), (-2.0 ** -40, 2.0 ** -112)])
def test_scores_next_to_nothing(scale, spread, window):
    """Small bf16 queries and scales over an 8-bit cache: all weights are alike, and hidden tokens have none."""
    c = Case([(200, 9), (3, 33), (0, 5), (700, 20)], 4, 2, 64, "bf16", "e4m3", window=window, scale=scale, spread=spread, seed=40)
    c.run().check()


def test_scores_of_zero_under_the_largest_scale():
    """Large bf16 queries whose products with the keys are 0, under a scale next to fp32's largest."""
    c = Case([(200, 9), (3, 33)], 4, 2, 64, "bf16", "e4m3", scale=3.0e38, seed=41)
    c.q.zero_()
    for h in range(4):
        c.q[:, 64 * h] = 2.0 ** 100
    c.k.view(torch.uint8)[..., 0] = 0
    c.run().check()
