"""The sign of zeros in 8-bit codes: a zero, or a value that rounds to zero,
keeps its sign, whatever the block's scale (the codes are those of the
correctly rounded quotient, bit for bit)."""

import numpy as np
import pytest
import torch

import sparse_moe_layer_latentmoe_amd as pkg
from oracle import operators as R

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F, B = torch.float32, torch.bfloat16


def values(rows, cols, seed, std):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, cols, generator=g) * std
    u = torch.rand(rows, cols, generator=g)
    x[u < 0.2] = -0.0
    x[u > 0.8] = 0.0
    x[(u > 0.4) & (u < 0.5)] *= -1e-5       # rounds to a zero of its sign
    return x


@pytest.mark.parametrize("dtype", [B, F])
@pytest.mark.parametrize("std", [1e-30, 1e-3, 1.0, 300.0, 1e30])
@pytest.mark.parametrize("cols", [128, 640, 131])
def test_activations(cols, std, dtype):
    x = values(9, cols, cols, std).to(dtype)
    q, s = pkg.quantize_fp8(x.to(DEV))
    want, scales = R.quantize_fp8(x.float().numpy())
    got = q.view(torch.uint8).cpu().numpy()
    assert np.array_equal(s.cpu().numpy(), scales)
    assert (want == 0x80).sum() > 100 and (want == 0).sum() > 100
    assert np.array_equal(got, want)


@pytest.mark.parametrize("dtype", [B, F])
@pytest.mark.parametrize("shape", [(128, 256), (144, 131)])
def test_weights(shape, dtype):
    w = values(*shape, 7, 0.02).to(dtype)
    q, s = pkg.quantize_fp8_weight(w.to(DEV))
    want, scales = R.quantize_fp8(w.float().numpy(), 128)
    assert np.array_equal(s.cpu().numpy(), scales)
    assert np.array_equal(q.view(torch.uint8).cpu().numpy(), want)
