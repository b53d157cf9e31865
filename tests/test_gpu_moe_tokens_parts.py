"""The sparse layer for a few tokens keeps its operands' 24 bits, whatever the
type of its result: where large values cancel, nothing but the result's own
rounding is lost.

One expert of weight 1 whose matrices hold 1, -1 and 0, so that every number on
the way is known.  An operand of 24 bits is the sum of three bf16 numbers (8
bits each); a sum of two such operands next to each other is exact in fp32, in
any order of their parts: every partial sum is a multiple of the operands' last
bit and at most twice their size.  What remains is the square's rounding, which
fp32 does the same way anywhere, and the result's: bits are compared."""

import numpy as np
import pytest
import torch

import sparse_moe_layer_latentmoe_amd as pkg

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F, B = torch.float32, torch.bfloat16
N = 256               # width and hidden width


def matrix(v, fmt):
    """(codes, scales) of a [1, N, N] matrix of 1, -1 and 0."""
    v = v[None].to(DEV)
    if fmt == "bf16":
        return v.to(B), None
    if fmt == "fp8":
        return v.to(torch.float8_e4m3fn), torch.ones(1, N // 128, N // 128, device=DEV)
    c = (2 * v.abs() + 8 * (v < 0)).to(torch.uint8)       # 1.0 is code 2
    return c[..., 0::2] | c[..., 1::2] << 4, torch.full((1, N, N // 32), 127, dtype=torch.uint8,
                                                        device=DEV)


def pairs(far):
    """Row i: column i minus column i + N / 2 (far: lines of different waves), or
    column 2 i minus 2 i + 1; the rows behind are 0."""
    m = torch.zeros(N, N)
    i = torch.arange(N // 2)
    m[i, i if far else 2 * i] = 1.0
    m[i, i + N // 2 if far else 2 * i + 1] = -1.0
    return m


def near(T, far, seed, bits):
    """x [T, N] of 24 bits whose pairs differ by 2^-bits of themselves."""
    g = torch.Generator().manual_seed(seed)
    a = 1.0 + torch.rand(T, N // 2, generator=g)
    b = a * (1.0 - 2.0 ** -bits * (1.0 + torch.rand(T, N // 2, generator=g)))
    return torch.cat([a, b], 1) if far else torch.stack([a, b], 2).flatten(1)


def run(x, up, down, fmt, out):
    (u, us), (d, ds) = matrix(up, fmt), matrix(down, fmt)
    y, idx, w = pkg.moe_tokens(pkg.make_router(1, 1), x.to(DEV), torch.ones(1, N, device=DEV), u, d,
                               up_scales=us, down_scales=ds, out_dtype=out)
    assert bool((w == 1).all()) and not bool(idx.any())
    return y.cpu()


def difference(v, far):
    v = v.numpy()
    h = v.shape[1] // 2
    d = (v[:, :h] - v[:, h:]) if far else (v[:, 0::2] - v[:, 1::2])
    assert np.array_equal(d.astype(np.float64), (v[:, :h].astype(np.float64) - v[:, h:]) if far else
                          (v[:, 0::2].astype(np.float64) - v[:, 1::2]))
    return np.concatenate([d, np.zeros_like(d)], 1)


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "mxfp4"])
@pytest.mark.parametrize("out", [F, B])
@pytest.mark.parametrize("far", [False, True])
@pytest.mark.parametrize("T", [1, 5, 6, 16])
def test_tokens_that_cancel(T, far, out, fmt):
    """u = x_a - x_b, y = u^2."""
    x = near(T, far, T, 12)
    u = difference(x, far)
    assert (u[:, :N // 2] > 0).all()
    want = torch.from_numpy(u * u).to(out)
    assert torch.equal(run(x, pairs(far), torch.eye(N), fmt, out), want)


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "mxfp4"])
@pytest.mark.parametrize("out", [F, B])
@pytest.mark.parametrize("far", [False, True])
@pytest.mark.parametrize("T", [1, 5, 6, 16])
def test_hidden_values_that_cancel(T, far, out, fmt):
    """u = x, y = x_a^2 - x_b^2 of the squares rounded to fp32."""
    x = near(T, far, 50 + T, 12)
    h = torch.from_numpy(x.numpy() * x.numpy())
    want = torch.from_numpy(difference(h, far)).to(out)
    assert torch.equal(run(x, torch.eye(N), pairs(far), fmt, out), want)
