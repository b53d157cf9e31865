"""The operators around the layer on the CPU: the C ABI refuses bad arguments
before any HIP call, the binding refuses tensors the kernels could not take,
and the oracle's gradients agree with central differences of its forward."""

import ctypes

import numpy as np
import pytest
import torch

import sparse_moe_layer_latentmoe_amd as pkg
from oracle import operators as R

FAKE = 0x10000000     # never dereferenced
INV, UNS, WS = pkg.LMOE_ERR_INVALID_ARG, pkg.LMOE_ERR_UNSUPPORTED, pkg.LMOE_ERR_WORKSPACE


@pytest.fixture(scope="module")
def lib():
    return pkg.load_library()


def at(i):
    return FAKE + (i << 32)


def route(lib, r, logits=at(0), lt=0, stride=None, bias=None, T=4, idx=at(1), w=at(2)):
    return lib.lmoe_route_logits(r, logits, lt, r.n_experts if stride is None else stride, bias, T,
                                 idx, w, None)


@pytest.mark.parametrize("kw,status", [
    (dict(n_experts=0), INV), (dict(top_k=0), INV), (dict(top_k=17), INV),
    (dict(n_experts=-4), INV), (dict(score=2), INV), (dict(n_group=3), INV),
    (dict(n_group=0), INV), (dict(n_group=4, topk_group=5), INV), (dict(topk_group=0), INV),
    (dict(n_group=4, topk_group=1, top_k=5), INV), (dict(group_score=0), INV),
    (dict(group_score=3), INV), (dict(n_group=16, topk_group=8, group_score=2), INV),
    (dict(scale=float("nan")), INV), (dict(n_experts=1025), UNS),
    (dict(n_experts=256, top_k=65), UNS),
    (dict(n_experts=1024, n_group=128, topk_group=8), UNS),
])
def test_router_settings_are_checked(lib, kw, status):
    base = dict(n_experts=16, top_k=4)
    base.update(kw)
    r = pkg.make_router(**base)
    assert route(lib, r) == status
    assert lib.lmoe_route_logits_backward(r, at(0), 0, 2048, at(1), at(2), 4, at(3), None) == status


def test_route_arguments_are_checked(lib):
    r = pkg.make_router(16, 4)
    assert lib.lmoe_route_logits(None, at(0), 0, 16, None, 4, at(1), at(2), None) == INV
    r2 = pkg.make_router(16, 4)
    r2.renormalise = 2
    assert route(lib, r2) == INV
    assert route(lib, r, T=0, logits=None, idx=None, w=None) == pkg.LMOE_OK
    for kw in (dict(logits=None), dict(idx=None), dict(w=None), dict(lt=2), dict(lt=-1),
               dict(stride=15), dict(T=-1), dict(logits=at(0) + 2), dict(bias=at(5) + 1),
               dict(idx=at(1) + 2), dict(w=at(0)), dict(idx=at(0) + 252), dict(w=at(1) + 60)):
        assert route(lib, r, **kw) == INV, kw
    assert route(lib, r, T=(1 << 22) + 1) == UNS
    back = lib.lmoe_route_logits_backward
    assert back(r, at(0), 0, 16, at(1), at(2), 0, None, None) == pkg.LMOE_OK
    for args in ((None, 0, 16, at(1), at(2), 4, at(3)), (at(0), 0, 16, None, at(2), 4, at(3)),
                 (at(0), 0, 16, at(1), None, 4, at(3)), (at(0), 0, 16, at(1), at(2), 4, None),
                 (at(0), 0, 16, at(1), at(2), 4, at(0)), (at(0), 0, 16, at(1), at(2), 4, at(2) - 8),
                 (at(0), 1, 16, at(1), at(2), 4, at(3) + 1)):
        assert back(r, *args, None) == INV, args


def norm_args(**kw):
    a = pkg.LmoeBlockNormArgs()
    for k, v in dict(h=at(0), y=at(1), h_stride=64, y_stride=64, pre_weight=at(2),
                     post_weight=at(3), res_scale=at(4), gate=at(5), gate_kind=1, h_type=0,
                     y_type=1, pre_type=1, post_type=1, res_scale_type=1, gate_type=1, T=3, D=64,
                     eps=1e-5).items():
        setattr(a, k, v)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), INV), (dict(D=0), INV), (dict(eps=0.0), INV), (dict(eps=float("inf")), INV),
    (dict(h=None), INV), (dict(h_stride=63), INV), (dict(y_stride=1), INV), (dict(h_type=2), INV),
    (dict(gate_type=-1), INV), (dict(gate_kind=4), INV), (dict(gate=None), INV),
    (dict(gate_kind=0), INV), (dict(y=None), INV), (dict(y=None, gate=None, gate_kind=0), INV),
    (dict(h=at(0) + 2), INV), (dict(post_weight=at(3) + 1), INV),
    (dict(D=16385, h_stride=16385, y_stride=16385), UNS), (dict(T=(1 << 22) + 1), UNS),
])
def test_block_norm_settings_are_checked(lib, kw, status):
    a = norm_args(**kw)
    assert lib.lmoe_block_norm(a, at(6), at(7), at(8), None) == status
    g = pkg.LmoeBlockNormGrads(at(9), None, at(10), None, None, None)
    assert lib.lmoe_block_norm_workspace_size(a, g) == 0
    assert lib.lmoe_block_norm_backward(a, at(8), at(6), at(7), g, at(11), 1 << 30, None) == status


def test_block_norm_outputs_are_checked(lib):
    a = norm_args()
    assert lib.lmoe_block_norm(None, at(6), at(7), None, None) == INV
    assert lib.lmoe_block_norm(norm_args(T=0), None, None, None, None) == pkg.LMOE_OK
    for out in ((None, at(7), None), (at(0), at(7), None), (at(6), at(1) + 8, None),
                (at(6), at(6) + 64, None), (at(6), at(7), at(5)), (at(6) + 2, at(7), None)):
        assert lib.lmoe_block_norm(a, *out, None) == INV, out
    G = pkg.LmoeBlockNormGrads
    g = G(at(9), at(10), at(11), at(12), at(13), at(14))
    need = lib.lmoe_block_norm_workspace_size(a, g)
    assert need >= 4 * 64 * 4
    assert lib.lmoe_block_norm_workspace_size(a, G(at(9), at(10), None, None, None, None)) == 0
    back = lib.lmoe_block_norm_backward
    assert back(a, at(8), None, at(7), g, None, need, None) == WS
    assert back(a, at(8), None, at(7), g, at(15), need - 1, None) == WS
    assert back(a, at(8), None, at(7), g, at(15) + 4, need, None) == WS
    assert back(a, at(8), None, at(7), None, at(15), need, None) == INV
    assert back(a, None, None, at(7), g, at(15), need, None) == INV
    assert back(a, at(8), None, at(7), g, at(9), need, None) == INV        # workspace on dh
    assert back(a, at(8), at(9), at(7), g, at(15), need, None) == INV      # dh_out on dh
    # a gradient of something that is not there
    for drop, want in (("pre_weight", 2), ("post_weight", 3), ("res_scale", 4)):
        only = [None] * 6
        only[want] = at(11)
        assert back(norm_args(**{drop: None}), at(8), None, at(7), G(*only), at(15), 1 << 30,
                    None) == INV, drop
    b = norm_args(gate=None, gate_kind=0)
    assert back(b, at(8), None, at(7), G(None, None, None, None, None, at(14)), at(15), 1 << 30,
                None) == INV
    c = norm_args(y=None, post_weight=None, gate=None, gate_kind=0)
    assert back(c, at(8), None, at(7), G(None, at(10), None, None, None, None), at(15), 1 << 30,
                None) == INV


def test_binding_refuses_tensors_it_cannot_pass():
    r = pkg.make_router(16, 4)
    x = torch.zeros(4, 16)
    with pytest.raises(ValueError, match="GPU"):
        pkg.route_logits(r, x)
    with pytest.raises(TypeError, match="dtype"):
        pkg.route_logits(r, x.half())
    with pytest.raises(TypeError, match="torch.Tensor"):
        pkg.route_logits(r, [[0.0]])
    with pytest.raises(ValueError, match="dimensions"):
        pkg.route_logits(r, torch.zeros(16))
    with pytest.raises(ValueError, match="rows"):
        pkg.route_logits(r, torch.zeros(16, 4).t())
    with pytest.raises(ValueError, match="rows"):
        pkg.route_logits(r, torch.zeros(1, 16).expand(4, 16))
    with pytest.raises(ValueError, match="GPU"):
        pkg.block_norm(x, x)
    with pytest.raises(TypeError, match="dtype"):
        pkg.block_norm(x.double(), x)


# ---- the oracle's own gradients ---------------------------------------------


def central(f, v, d, eps=1e-6):
    """d/dv of sum(f(v) * d) by central differences."""
    out = np.zeros_like(v)
    for i in np.ndindex(v.shape):
        hi, lo = v.copy(), v.copy()
        hi[i] += eps
        lo[i] -= eps
        out[i] = ((f(hi) - f(lo)) * d).sum() / (2 * eps)
    return out


@pytest.mark.parametrize("softmax", [False, True])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_gradient_against_differences(softmax, renorm):
    g = np.random.default_rng(1)
    l, bias, dw = g.normal(size=(3, 12)), g.normal(size=12) * 0.1, g.normal(size=(3, 4))
    kw = dict(softmax=softmax, renorm=renorm, scale=2.5)
    idx, _ = R.route(l, bias, 4, n_group=3, topk_group=2, **kw)

    def f(v):
        s = np.take_along_axis(R.route_scores(v, softmax), idx, 1)
        return 2.5 * (s / (s.sum(1, keepdims=True) + 1e-20) if renorm else s)

    # differences: eps^2 terms and 1e-16 / eps cancellation, both below 1e-8 here
    assert np.allclose(R.route_backward(l, idx, dw, **kw)[0], central(f, l, dw), atol=1e-7)


@pytest.mark.parametrize("gate_shape", [None, (7,), (4, 1), (4, 7)])
@pytest.mark.parametrize("post", [True, False])
def test_block_norm_gradient_against_differences(gate_shape, post):
    g = np.random.default_rng(2)
    T, D = 4, 7
    v = dict(h=g.normal(size=(T, D)), y=g.normal(size=(T, D)), pre=g.normal(size=D),
             post=g.normal(size=D) if post else None,
             gate=None if gate_shape is None else g.normal(size=gate_shape),
             alpha=g.normal(size=D))
    dh, dx = g.normal(size=(T, D)), g.normal(size=(T, D))
    got = R.block_norm_backward(v["h"], v["y"], dh, dx, v["pre"], v["post"], v["gate"],
                                v["alpha"], 1e-3)
    names = dict(h="dh", y="dy", pre="dpre_weight", post="dpost_weight", gate="dgate",
                 alpha="dres_scale")
    for n, gn in names.items():
        if v[n] is None:
            assert gn not in got
            continue

        def f(u):
            w = dict(v)
            w[n] = u
            a, b, _, _ = R.block_norm(w["h"], w["y"], w["pre"], w["post"], w["gate"],
                                      w["alpha"], 1e-3)
            return np.stack([a, b])

        want = central(f, v[n], np.stack([dh, dx]))
        assert np.allclose(got[gn][0], want, atol=1e-6), n
