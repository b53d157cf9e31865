"""The sparse layer for a few tokens where experts have more rows than are taken
at a time (five in fp32; all of them in bf16 going up): every row count beside
the borders, in each format, against float64."""

import pytest
import torch

import sparse_moe_layer_latentmoe_amd as pkg
from test_gpu_moe_tokens import DEV, FORMATS, Layer, rand

pytestmark = pytest.mark.gpu
F, B = torch.float32, torch.bfloat16


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("T", [5, 6, 10, 11, 15, 16])
def test_shared_expert_and_crowded_experts(T, swiglu, fmt):
    layer = Layer(7, 3, 384, 256, fmt, swiglu, 384, seed=T, score=pkg.SCORE_SOFTMAX)
    layer.bias[[1, 4]] = 3.0              # two that every token takes
    for x, out in ((B, B), (F, F), (B, F), (F, B)):
        layer.check(rand(T, 384, seed=T, dtype=x), out=out)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("x", [F, B])
def test_row_counts_side_by_side(x, fmt):
    """Expert e has e rows: a token takes the experts above its own number."""
    T = K = 16
    layer = Layer(33, K, 256, 128, fmt, seed=3, bias=True)
    layer.bias = torch.zeros(33, device=DEV)
    # logits of weight 8 on one column a token: expert e (1 .. 16) in the first e tokens,
    # and experts 17 .. 32 for what is left of the 16
    tok = torch.zeros(T, 256)
    gate = torch.zeros(33, 256)
    for t in range(T):
        tok[t, t] = 1.0
        for e in range(1, 17):
            gate[e, t] = 8.0 if t < e else -8.0
        gate[17:, t] = torch.linspace(-1, 1, 16)
    layer.gate = gate.to(DEV)
    tok[:, 16:] = torch.randn(T, 240, generator=torch.Generator().manual_seed(5))
    y = layer.check(tok.to(x).to(DEV), out=F)
    idx = layer(tok.to(x).to(DEV), F)[1]
    count = torch.bincount(idx.flatten(), minlength=33)
    assert count[1:17].tolist() == list(range(1, 17)) and y.shape == (T, 256)


@pytest.mark.parametrize("fmt", FORMATS)
def test_many_pairs(fmt):
    """Top-64: the longest lists, with more experts than are routed in the kernel."""
    for E in (200, 1024):
        layer = Layer(E, 64, 128, 128, fmt, seed=E, S=128)
        for x in (B, F):
            layer.check(rand(16, 128, seed=E, dtype=x), out=F)


@pytest.mark.parametrize("x", [F, B])
def test_a_token_is_the_same_in_any_company(x):
    """One token's row, alone, among five and among sixteen that take its experts."""
    layer = Layer(6, 6, 512, 384, "mxfp4", True, 256, seed=8, score=pkg.SCORE_SOFTMAX)
    t = rand(16, 512, seed=9, dtype=x)
    y = layer(t, F)[0]
    for n in (5, 6, 11):
        assert torch.equal(layer(t[:n], F)[0], y[:n])
