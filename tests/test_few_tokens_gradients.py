"""The 4-bit product and the layer for a few tokens have no gradient: every
argument that could require one is refused while autograd records (on the CPU:
the refusal comes before any look at the device)."""

import pytest
import torch

import sparse_moe_layer_latentmoe_amd as pkg

B = torch.bfloat16


def layer(**leaf):
    """A call of FP8 experts with a shared one; `leaf` replaces arguments."""
    e4, s = torch.float8_e4m3fn, torch.ones(2, 1, 1)
    a = dict(x=torch.zeros(1, 128), gate=torch.zeros(2, 128), up=torch.zeros(2, 128, 128).to(e4),
             down=torch.zeros(2, 128, 128).to(e4), bias=torch.zeros(2), up_scales=s, down_scales=s,
             shared_up=torch.zeros(128, 128).to(e4), shared_down=torch.zeros(128, 128).to(e4),
             shared_up_scales=s[0], shared_down_scales=s[0])
    a.update(leaf)
    return pkg.moe_tokens(pkg.make_router(2, 1), **a)


@pytest.mark.parametrize("name,shape", [
    ("x", (1, 128)), ("gate", (2, 128)), ("bias", (2,)), ("up_scales", (2, 1, 1)),
    ("down_scales", (2, 1, 1)), ("shared_up_scales", (1, 1)), ("shared_down_scales", (1, 1))])
def test_layer_refuses_what_needs_a_gradient(name, shape):
    leaf = torch.ones(shape, requires_grad=True)
    with pytest.raises(ValueError, match="gradient"):
        layer(**{name: leaf})
    # without autograd the next check speaks
    with torch.no_grad(), pytest.raises(ValueError, match="GPU"):
        layer(**{name: leaf})


@pytest.mark.parametrize("name", ["up", "down"])
def test_layer_refuses_weights_that_need_a_gradient(name):
    w = torch.zeros(2, 128, 128, dtype=B, requires_grad=True)
    with pytest.raises(ValueError, match="gradient"):
        layer(**{name: w})


def test_product_refuses_an_output_that_needs_a_gradient():
    x, s = torch.zeros(4, 64, dtype=torch.uint8), torch.zeros(4, 4, dtype=torch.uint8)
    out = torch.zeros(4, 4, requires_grad=True)
    with pytest.raises(ValueError, match="gradient"):
        pkg.mxfp4_matmul(x, s, x, s, out=out)
    with torch.no_grad(), pytest.raises(ValueError, match="GPU"):
        pkg.mxfp4_matmul(x, s, x, s, out=out)
