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


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("scale", [2.5, 1e25])
@pytest.mark.parametrize("size", [1.0, 1e10])
def test_scores_near_nothing_under_large_factors(size, scale, score):
    """Selected scores whose sum is about the 1e-20 beside it, and rows with
    nothing available: the factor scale / sum is beyond fp32, the weights and
    gradients are not.  Bounds: 2^-17 for a weight (its score and the quotient);
    for a gradient 2^-15 of its terms' magnitudes."""
    E, K = 96, 8
    l = torch.full((7, E), -3.0)
    l[0] = float("-inf")
    l[1, 8:] = float("-inf")
    for t in range(1, 7):                       # scores of 1e-28 to 1e-19
        l[t, :8] = torch.linspace(-64.0, -44.0, 8) + t
    l[6, 2:5] = float("nan")
    bias = torch.zeros(E)
    bias[:8] = 4.0
    l, bias = l.to(DEV), bias.to(DEV)
    softmax = score == "softmax"
    r = pkg.make_router(E, K, pkg.SCORE_SOFTMAX if softmax else pkg.SCORE_SIGMOID, scale=scale)
    idx, w = pkg.route_logits(r, l, bias)
    want, want_w = R.route(exact(l), exact(bias), K, softmax, scale=scale)
    assert np.array_equal(idx.cpu().numpy(), want)
    assert np.all(np.abs(exact(w) - want_w) <= 2.0 ** -17 * np.abs(want_w))
    gen = torch.Generator().manual_seed(4)
    dw = (torch.randn(7, K, generator=gen) * size).to(DEV)
    dl = pkg.route_logits_backward(r, l, idx, dw)
    ref, mag = R.route_backward(exact(l), want, exact(dw), softmax, scale=scale)
    assert np.all(np.abs(exact(dl) - ref) <= 2.0 ** -15 * mag + 2.0 ** -126)
    assert not dl[0].any()
