"""Routing from given logits on the GPU against the float64 oracle: the
selection exactly (it is defined on 64-bit values), weights and gradients
within bounds that follow from the kernel's fp32 steps.

Bounds.  A score: exp is within 1 ulp and its argument is rounded by
2^-24 |l - max| (at most 2^-19.4 relative where a score is above e^-24, the
smallest the random inputs here select), additions of up to 1024 positive
terms in a tree of 16 + 6 steps add 22 half-ulps, two products and a quotient
three more: 2^-18 relative in all.  A weight: score / sum of scores: 2^-17.
A gradient: products of three such factors and one difference whose terms'
magnitudes the oracle adds up: 2^-15 of that; then the rounding to the
logits' type (2^-8 for bf16)."""

import numpy as np
import pytest
import torch

import sparse_moe_layer_latentmoe_amd as pkg
from oracle import operators as R

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def tensor(v, dtype=torch.float32):
    return torch.from_numpy(np.asarray(v, np.float32)).to(DEV, dtype)


def exact(t):
    return t.double().cpu().numpy()


def run(l, K, bias=None, dw=None, score="sigmoid", n_group=1, topk_group=1, group_score=2,
        renorm=True, scale=1.0):
    """Kernel and oracle on the values of `l` (a GPU tensor); checks both directions."""
    T, E = l.shape
    r = pkg.make_router(E, K, pkg.SCORE_SOFTMAX if score == "softmax" else pkg.SCORE_SIGMOID,
                        n_group, topk_group, group_score, renorm, scale)
    idx, w = pkg.route_logits(r, l, bias)
    kw = dict(softmax=score == "softmax", renorm=renorm, scale=scale)
    b = None if bias is None else exact(bias)
    want_idx, want_w = R.route(exact(l), b, K, n_group=n_group, topk_group=topk_group,
                               group_score=group_score, **kw)
    assert np.array_equal(idx.cpu().numpy(), want_idx)
    # scores below the smallest normal fp32 number keep its absolute spacing
    assert np.all(np.abs(exact(w) - want_w) <= 2.0 ** -17 * np.abs(want_w) + abs(scale) * 2.0 ** -126)
    g = torch.Generator().manual_seed(5)
    dw = torch.randn(T, K, generator=g).to(DEV)
    dl = pkg.route_logits_backward(r, l, idx, dw)
    want, mag = R.route_backward(exact(l), want_idx, exact(dw), **kw)
    unit = torch.finfo(l.dtype).eps / 2 if l.dtype == torch.bfloat16 else 0.0
    err = np.abs(exact(dl) - want)
    assert np.all(err <= 2.0 ** -15 * mag + unit * np.abs(want) + 2.0 ** -126), err.max()
    return idx, w, dl


def logits(T, E, seed, dtype=torch.float32, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(T, E, generator=g) * std).to(dtype).to(DEV)


def bias_of(E, seed, std=0.1):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(E, generator=g) * std).to(DEV)


@pytest.mark.parametrize("T", [1, 3, 65])
@pytest.mark.parametrize("E,K", [(1, 1), (8, 2), (63, 7), (64, 64), (65, 9), (130, 22), (512, 22),
                                 (509, 8), (1024, 64)])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_sizes(T, E, K, score):
    run(logits(T, E, T + E), K, bias_of(E, 3), score=score, scale=5.0)
    run(logits(T, E, T + E + 1, torch.bfloat16), K, score=score, renorm=False)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("bias", [True, False])
@pytest.mark.parametrize("E,K,groups,kept,best", [
    (512, 22, 8, 4, 2), (512, 6, 64, 3, 1), (40, 8, 4, 2, 1), (60, 5, 20, 4, 2), (96, 9, 3, 3, 2),
    (1024, 30, 2, 1, 2), (16, 4, 16, 4, 1)])
def test_groups(E, K, groups, kept, best, bias, score):
    run(logits(70, E, E), K, bias_of(E, 4) if bias else None, score=score, n_group=groups,
        topk_group=kept, group_score=best)


def test_equal_scores_go_to_the_lower_id():
    l = torch.zeros(5, 200, device=DEV)
    idx, w, _ = run(l, 6)
    assert np.array_equal(idx.cpu().numpy(), np.tile(np.arange(6), (5, 1)))
    run(l, 6, torch.zeros(200, device=DEV))
    run(l, 6, torch.zeros(200, device=DEV), n_group=8, topk_group=3)
    # bf16 logits take few values, so most borders are ties
    run((logits(64, 512, 9) * 4).round().div(4).to(torch.bfloat16), 22)
    run((logits(64, 512, 9) * 4).round().div(4).to(torch.bfloat16), 22,
        torch.zeros(512, device=DEV), n_group=8, topk_group=4)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_borders_closer_than_an_fp32_score(score):
    """Biased scores that differ by less than an fp32 ulp, and in the order
    opposite to the ids: only their 64-bit values tell them apart."""
    E, K = 192, 8
    l = logits(40, E, 11)
    s = R.route_scores(exact(l), score == "softmax")
    # a bias that levels token t's scores up to its own fp32 rounding
    for t in range(0, 40, 8):
        b = tensor(0.5 - s[t])
        run(l, K, b, score=score)
        run(l, K, b, score=score, n_group=6, topk_group=2)


def test_scores_that_saturate():
    l = torch.linspace(12.0, 36.0, 256, device=DEV).repeat(3, 1)[:, torch.randperm(
        256, generator=torch.Generator().manual_seed(0))]
    run(l, 16)                                      # ordered by the logits themselves
    run(l, 16, bias_of(256, 2, 1e-9))
    run(-l, 16, n_group=4, topk_group=2)            # group sums of tiny scores
    run(l * 40, 4, score="softmax", renorm=False)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_unavailable_experts(score):
    l = logits(9, 96, 13)
    l[0] = float("-inf")                             # nothing available
    l[1, 5:] = float("nan")                          # fewer than K
    l[2, ::2] = float("-inf")
    l[3, :3] = float("inf")
    l[4] = torch.finfo(torch.float32).min
    l[5, 40:] = torch.finfo(torch.float32).min
    l[6, 10] = float("inf")
    for bias in (None, bias_of(96, 6, 3.0)):
        idx, w, dl = run(l, 8, bias, score=score)
        assert torch.equal(idx[0].cpu(), torch.arange(8, dtype=torch.int32))
        assert not w[0].any() and not dl[0].any()
        assert not dl[2, ::2].any()
        run(l, 8, bias, score=score, n_group=4, topk_group=2)


def test_strided_rows_other_streams_and_no_rows():
    wide = logits(33, 300, 17, torch.bfloat16)
    a = run(wide[:, 7:107], 9)
    b = run(wide[:, 7:107].contiguous(), 9)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    r = pkg.make_router(100, 9)
    x = wide[:, 7:107]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    i1, w1 = pkg.route_logits(r, x, stream=side)
    i2, w2 = pkg.route_logits(r, x, stream=side.cuda_stream)
    side.synchronize()
    assert torch.equal(i1, a[0]) and torch.equal(w1, a[1])
    assert torch.equal(i2, a[0]) and torch.equal(w2, a[1])
    e = pkg.route_logits(r, x[:0])
    assert e[0].shape == (0, 9) and e[1].shape == (0, 9)
    assert pkg.route_logits_backward(r, x[:0], *e).shape == (0, 100)


def test_backward_ignores_bad_ids_and_adds_equal_ones():
    l = logits(4, 70, 19)
    idx = torch.tensor([[3, 3, 3, 9], [-1, 70, 5, 2 ** 30], [69, 0, 69, 0], [1, 2, 3, 4]],
                       dtype=torch.int32, device=DEV)
    dw = logits(4, 4, 20)
    for score, renorm in (("sigmoid", True), ("sigmoid", False), ("softmax", False)):
        soft = score == "softmax"
        r = pkg.make_router(70, 4, pkg.SCORE_SOFTMAX if soft else pkg.SCORE_SIGMOID,
                            renormalise=renorm)
        got = exact(pkg.route_logits_backward(r, l, idx, dw))
        want, mag = R.route_backward(exact(l), idx.cpu().numpy(), exact(dw), softmax=soft,
                                     renorm=renorm)
        assert np.all(np.abs(got - want) <= 2.0 ** -15 * mag + 1e-37)


def test_rows_further_apart_than_32_bits():
    r = pkg.make_router(70, 4)
    l, dw = logits(2, 70, 26), logits(2, 4, 27)
    far = torch.empty(2, 2 ** 31, device=DEV)[:, :70]
    far.copy_(l)
    idx, w = pkg.route_logits(r, l)
    i2, w2 = pkg.route_logits(r, far)
    assert torch.equal(idx, i2) and torch.equal(w, w2)
    assert torch.equal(pkg.route_logits_backward(r, l, idx, dw),
                       pkg.route_logits_backward(r, far, idx, dw))


@pytest.mark.parametrize("gap", [0.0, 2.0 ** -24, 2.0 ** -22, 2.0 ** -20])
@pytest.mark.parametrize("softmax", [False, True])
def test_many_keys_next_to_the_border(gap, softmax):
    """More than 64 biased scores within the scores' error of each other, a few
    of them (which fit one a lane), and a border between equal ones."""
    l = logits(6, 512, 28)
    for t, n in enumerate((2, 20, 40, 64, 100, 512)):
        pick = torch.randperm(512, generator=torch.Generator().manual_seed(t))[:n].to(DEV)
        l[t, pick] = 2.0 + gap * torch.randint(0, 3, (n,), generator=torch.Generator()
                                               .manual_seed(t + 9)).to(DEV)
    b = bias_of(512, 29)
    b[::2] = 0.25                                      # equal biases of half the experts
    for K, kw in ((8, {}), (22, {}), (22, dict(n_group=8, topk_group=4)), (64, {})):
        r = pkg.make_router(512, K, pkg.SCORE_SOFTMAX if softmax else pkg.SCORE_SIGMOID, **kw)
        idx, _ = pkg.route_logits(r, l, b)
        want, _ = R.route(exact(l), exact(b), K, softmax=softmax, **kw)
        assert np.array_equal(idx.cpu().numpy(), want)


def test_replayed_from_a_graph():
    r = pkg.make_router(512, 22, n_group=8, topk_group=4, scale=5.0)
    l, b, dw = logits(32, 512, 23), bias_of(512, 24), logits(32, 22, 25)
    static = l.clone()
    pkg.route_logits(r, static, b)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        idx, w = pkg.route_logits(r, static, b)
        dl = pkg.route_logits_backward(r, static, idx, dw)
    for seed in range(3):
        static.copy_(logits(32, 512, 30 + seed))
        g.replay()
        torch.cuda.synchronize()
        i2, w2 = pkg.route_logits(r, static, b)
        d2 = pkg.route_logits_backward(r, static, i2, dw)
        assert torch.equal(idx, i2) and torch.equal(w, w2) and torch.equal(dl, d2)
