"""Routing at the ends of its arguments' ranges, against the float64 oracle."""

import numpy as np
import pytest
import torch

import sparse_moe_layer_latentmoe_amd as pkg
from oracle import operators as R

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
MAX = float(np.finfo(np.float32).max)


def exact(t):
    return t.double().cpu().numpy()


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("best", [1, 2])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_groups_whose_scores_pass_fp32(sign, best, score):
    """Biases near the largest finite number: the sum of two scores of a group
    is beyond fp32, its value in 64 bits orders the groups."""
    E, G, K = 64, 8, 6
    g = np.random.default_rng(1)
    bias = sign * MAX * (0.55 + 0.4 * np.repeat(g.permutation(G) / G, E // G))
    bias[::3] *= 0.98
    bias = torch.from_numpy(bias.astype(np.float32)).to(DEV)
    gen = torch.Generator().manual_seed(2)
    l = torch.randn(9, E, generator=gen).to(DEV)
    softmax = score == "softmax"
    r = pkg.make_router(E, K, pkg.SCORE_SOFTMAX if softmax else pkg.SCORE_SIGMOID, G, 3, best)
    idx, w = pkg.route_logits(r, l, bias)
    want, want_w = R.route(exact(l), exact(bias), K, softmax, G, 3, best)
    assert np.array_equal(idx.cpu().numpy(), want)
    # a score's and the quotient's bound: 2^-17 relative
    assert np.all(np.abs(exact(w) - want_w) <= 2.0 ** -17 * np.abs(want_w))
