"""MXFP4 scale bytes at the ends of their range in the layer for a few tokens:
0 is 2^-127, 254 is 2^127, and 255 is NaN, as in the products and the way back."""

import pytest
import torch

import sparse_moe_layer_latentmoe_amd as pkg

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F, U8 = torch.float32, torch.uint8
N = 128


def run(T, h, codes, scales, where="down"):
    """y [T, N] of one expert: hidden values h (a square of a power of 2), every
    down code `codes` in column 40 of row 5 (its block's scale `scales`), 1 in
    column 0 of the other rows."""
    up = torch.zeros(1, N, N // 2, dtype=U8, device=DEV)
    up[:, :, 0] = 2                      # 1.0 times the first value
    down = torch.zeros(1, N, N // 2, dtype=U8, device=DEV)
    down[:, :, 0] = 2
    down[:, 5, 0] = 0
    down[:, 5, 20] = codes
    us = torch.full((1, N, N // 32), 127, dtype=U8, device=DEV)
    ds = us.clone()
    (ds if where == "down" else us)[:, 5, 1] = scales
    x = torch.zeros(T, N, device=DEV)
    x[:, 0] = h ** 0.5
    y, _, w = pkg.moe_tokens(pkg.make_router(1, 1), x, torch.ones(1, N, device=DEV), up, down,
                             up_scales=us, down_scales=ds, out_dtype=F)
    assert bool((w == 1).all())
    return y


@pytest.mark.parametrize("T", [1, 6])
@pytest.mark.parametrize("code,value", [(1, 0.5), (2, 1.0), (7, 6.0), (10, -1.0)])
@pytest.mark.parametrize("byte", [0, 1, 2, 126, 127, 253, 254])
def test_every_scale(byte, code, value, T):
    h = 2.0 ** 40 if byte < 100 else 2.0 ** -40
    y = run(T, h, code, byte)
    want = torch.full((T, N), h, device=DEV)
    want[:, 5] = value * h * 2.0 ** (byte - 127)     # a power of 2 times 1 or 1.5
    if abs(value) * 2.0 ** (byte - 127) > torch.finfo(F).max:
        # 6 2^126 is 1.5 2^128, above fp32's and bf16's largest, 2^128 (1 - 2^-24) and
        # 2^128 (1 - 2^-8): the weight is infinite, and times the 0 that h, a bf16
        # number, leaves for its further parts it is NaN
        assert not bool(y[:, 5].isfinite().any())
        y[:, 5] = want[:, 5]
    assert torch.equal(y, want)


@pytest.mark.parametrize("T", [1, 6])
@pytest.mark.parametrize("code", [0, 2, 10])
def test_a_scale_that_is_not_a_number(code, T):
    y = run(T, 4.0, code, 255)
    rest = torch.arange(N, device=DEV) != 5
    assert bool(y[:, 5].isnan().all()) and bool((y[:, rest] == 4.0).all())
    # in the projection up: the hidden value, and with it the tokens' rows
    assert bool(run(T, 4.0, code, 255, "up").isnan().all())


def test_an_expert_that_is_not_used_does_not_matter():
    up = torch.full((3, N, N // 2), 0x22, dtype=U8, device=DEV)
    s = torch.full((3, N, N // 32), 120, dtype=U8, device=DEV)
    gate = torch.zeros(3, N, device=DEV)
    gate[1] = 1.0
    x = torch.ones(2, N, device=DEV)
    call = lambda: pkg.moe_tokens(pkg.make_router(3, 1), x, gate, up, up, up_scales=s,  # noqa: E731
                                  down_scales=s, out_dtype=F)[0]
    want = call()
    s[0] = s[2] = 255
    assert torch.equal(call(), want) and bool(want.isfinite().all())
