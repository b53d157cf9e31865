"""The sparse layer for a few tokens where a work-group waits in vain for hidden
rows: the number of its looks is set to next to nothing from the host, so that
every wait ends at once.  What it then adds to y is NaN, and nothing else is."""

import ctypes

import pytest
import torch

import sparse_moe_layer_latentmoe_amd as pkg

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F, B = torch.float32, torch.bfloat16


@pytest.fixture
def looks():
    """Sets the number of looks (lmoe::moe_tokens_looks) for one test."""
    n = ctypes.c_int.in_dll(pkg.load_library(), "_ZN4lmoe16moe_tokens_looksE")
    was = n.value
    assert was >= 1 << 20

    def put(v):
        n.value = was if v is None else v

    yield put
    n.value = was


def layer(T, E, D, H, S, out, swiglu):
    g = torch.Generator().manual_seed(T)

    def rand(*s, dtype=B, std=0.05):
        return (torch.randn(*s, generator=g) * std).to(dtype).to(DEV)

    two = 2 if swiglu else 1
    x, gate = rand(T, D, std=1.0), rand(E, D, dtype=F)
    up, down = rand(E, two * H, D), rand(E, D, H)
    sh = dict(shared_up=rand(two * S, D), shared_down=rand(D, S)) if S else {}
    return lambda: pkg.moe_tokens(pkg.make_router(E, 3), x, gate, up, down, out_dtype=out,
                                  activation=pkg.ACT_SWIGLU if swiglu else pkg.ACT_RELU2, **sh)


@pytest.mark.parametrize("out", [F, B])
@pytest.mark.parametrize("T,E,D,H,S", [(1, 16, 256, 384, 0), (6, 40, 512, 1024, 128),
                                       (16, 6, 1024, 512, 1024)])
def test_rows_waited_for_in_vain_are_nan(T, E, D, H, S, out, looks):
    call = layer(T, E, D, H, S, out, T == 6)
    want = call()
    assert bool(want[0].isfinite().all())
    looks(0)
    y, idx, w = call()
    torch.cuda.synchronize()
    assert bool(y.isnan().all())
    assert torch.equal(idx, want[1]) and torch.equal(w, want[2])
    for n in (1, 2, 5):                  # some are there in time
        looks(n)
        y, idx, w = call()
        torch.cuda.synchronize()
        assert torch.equal(torch.where(y.isnan(), want[0], y), want[0])
        assert torch.equal(idx, want[1]) and torch.equal(w, want[2])
    looks(None)
    assert all(torch.equal(a, b) for a, b in zip(call(), want))
