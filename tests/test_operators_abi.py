"""The operators around the layer on the CPU: the C ABI refuses bad arguments
before any HIP call, the binding refuses tensors the kernels could not take,
and the oracle's gradients agree with central differences of its forward."""

import ctypes

import numpy as np
import pytest
import torch

import lmoe_inputs as li
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


@pytest.mark.parametrize("T,D", [((1 << 22) - 1, 8192), (1, 16384), (1 << 22, 8)])
def test_block_norm_sizes_at_their_limits(lib, T, D):
    a = norm_args(T=T, D=D, h_stride=D, y_stride=D, h=None)   # refused for h, not for its size
    assert lib.lmoe_block_norm(a, at(6), at(7), None, None) == (UNS if T >> 22 else INV)


def test_quantiser_arguments_are_checked(lib):
    q = lib.lmoe_quantize_fp8
    base = dict(x=at(0), t=1, rows=4, cols=200, stride=200, codes=at(1), scales=at(2))

    def call(**kw):
        v = {**base, **kw}
        return q(v["x"], v["t"], v["rows"], v["cols"], v["stride"], v["codes"], v["scales"], None)

    assert call(rows=0, x=None, codes=None, scales=None) == pkg.LMOE_OK
    for kw in (dict(x=None), dict(codes=None), dict(scales=None), dict(t=2), dict(t=-1),
               dict(rows=-1), dict(cols=0), dict(stride=199), dict(x=at(0) + 1),
               dict(scales=at(2) + 2), dict(codes=at(0) + 1599), dict(scales=at(1) + 796),
               dict(t=0, x=at(0) + 2), dict(codes=at(2) + 28)):
        assert call(**kw) == INV, kw
    assert call(rows=1 << 27) == UNS                   # 2^28 blocks
    assert call(rows=1 << 40, cols=1, stride=1) == UNS
    assert call(stride=(1 << 31) + 1) == UNS
    qw = lib.lmoe_quantize_fp8_weight
    assert qw(None, 1, 0, 64, 64, None, None, None) == pkg.LMOE_OK
    for args in ((None, 1, 2, 64, 64, at(1), at(2)), (at(0), 1, 2, 64, 64, None, at(2)),
                 (at(0), 1, 2, 64, 64, at(1), None), (at(0), 3, 2, 64, 64, at(1), at(2)),
                 (at(0), 1, -1, 64, 64, at(1), at(2)), (at(0), 1, 2, 0, 64, at(1), at(2)),
                 (at(0), 1, 2, 64, 0, at(1), at(2)), (at(0) + 1, 1, 2, 64, 64, at(1), at(2)),
                 (at(0), 1, 2, 64, 64, at(0) + 16383, at(2)),
                 (at(0), 1, 2, 64, 64, at(1), at(1) + 8188)):
        assert qw(*args, None) == INV, args
    assert qw(at(0), 1, 1 << 22, 129, 129, at(1), at(2), None) == UNS   # 2^24 blocks


def mm_args(**kw):
    a = pkg.LmoeFp8MatmulArgs()
    for k, v in dict(x=at(0), x_scales=at(1), w=at(2), w_scales=at(3), rows=None, offsets=None,
                     y=at(4), y_type=1, n_groups=0, M=40, x_rows=40, N=256, K=1024).items():
        setattr(a, k, v)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("kw,status", [
    (dict(M=-1), INV), (dict(N=0), INV), (dict(K=0), INV), (dict(n_groups=-1), INV),
    (dict(x_rows=0), INV), (dict(y_type=2), INV), (dict(x=None), INV), (dict(x_scales=None), INV),
    (dict(w=None), INV), (dict(w_scales=None), INV), (dict(y=None), INV),
    (dict(x=at(0) + 8), INV), (dict(w=at(2) + 4), INV), (dict(y=at(4) + 8), INV),
    (dict(w_scales=at(3) + 2), INV), (dict(rows=at(5) + 2), INV), (dict(x_rows=39), INV),
    (dict(offsets=at(5)), INV), (dict(n_groups=3), INV), (dict(y=at(0) + 1024), INV),
    (dict(y=at(2) + (1 << 18) - 16), INV), (dict(y=at(1) - 16), INV),
    (dict(rows=at(4) + 32), INV), (dict(N=250), UNS), (dict(K=1000), UNS), (dict(K=65664), UNS),
    (dict(N=(1 << 20) + 16), UNS), (dict(M=(1 << 24) + 1, x_rows=1 << 25), UNS),
    (dict(n_groups=1025, offsets=at(5)), UNS),
    (dict(rows=at(5), x_rows=1 << 21), UNS)])
def test_product_arguments_are_checked(lib, kw, status):
    a = mm_args(**kw)
    assert lib.lmoe_fp8_matmul_workspace_size(a) == 0
    assert lib.lmoe_fp8_matmul(a, at(6), 1 << 30, None) == status


def test_product_workspace_is_checked(lib):
    size, mm = lib.lmoe_fp8_matmul_workspace_size, lib.lmoe_fp8_matmul
    assert mm(None, None, 0, None) == INV and size(None) == 0
    assert size(mm_args(M=0)) == 0 and mm(mm_args(M=0, x=None), None, 0, None) == pkg.LMOE_OK
    assert size(mm_args(M=5)) == 0                     # one pass over the weights
    split = mm_args(M=150, x_rows=150, N=2048, K=8192)  # few tiles: k is split
    grouped = mm_args(n_groups=3, offsets=at(5))
    for a in (split, grouped):
        need = size(a)
        assert need > 0
        assert mm(a, None, need, None) == WS
        assert mm(a, at(6), need - 1, None) == WS
        assert mm(a, at(6) + 8, need, None) == WS
        assert mm(a, at(0), need, None) == INV         # on x
        assert mm(a, at(4), need, None) == INV         # on y
    # a part's sums are fp32 [M, N]
    assert size(split) % (150 * 2048 * 4) == 0


def test_fp8_layer_settings_are_checked(lib):
    sh = li.LayerShape(256, 128, 16, 4, 256, 512, 5.0)

    def create(c, **kw):
        w = pkg.LmoeWeights()
        for name in ("fc1_latent", "router", "router_bias", "fc2_latent", "shared_up",
                     "shared_down", "expert_up_fp8", "expert_up_fp8_scale", "expert_down_fp8",
                     "expert_down_fp8_scale"):
            setattr(w, name, kw.get(name, FAKE))
        h = ctypes.c_void_p()
        return lib.lmoe_create(c, w, FAKE, 1 << 40, ctypes.byref(h))

    c = pkg.make_config(sh, 64, expert_format=pkg.EXPERTS_FP8)
    assert 0 < pkg.workspace_size(c) < pkg.workspace_size(pkg.make_config(sh, 64)) + (1 << 16)
    for name in ("expert_up_fp8", "expert_up_fp8_scale", "expert_down_fp8",
                 "expert_down_fp8_scale"):
        assert create(c, **{name: None}) == INV
        assert create(c, **{name: FAKE + 8}) == INV
    for bad in (li.LayerShape(256, 192, 16, 4, 256, 512, 5.0),
                li.LayerShape(256, 128, 16, 4, 320, 512, 5.0)):
        assert create(pkg.make_config(bad, 64, expert_format=pkg.EXPERTS_FP8)) == UNS
    # latent rows past 2 GiB
    long = li.LayerShape(256, 2048, 16, 4, 256, 512, 5.0)
    assert create(pkg.make_config(long, 1 << 20, expert_format=pkg.EXPERTS_FP8)) == UNS


def test_fp8_weight_specs():
    spec = pkg.weight_specs(li.FULL, pkg.EXPERTS_FP8)
    e4m3, f32 = torch.float8_e4m3fn, torch.float32
    assert "expert_up" not in spec and "expert_up_mxfp4" not in spec
    assert spec["expert_up_fp8"] == ((512, 5120, 2048), e4m3)
    assert spec["expert_up_fp8_scale"] == ((512, 40, 16), f32)
    assert spec["expert_down_fp8"] == ((512, 2048, 5120), e4m3)
    assert spec["expert_down_fp8_scale"] == ((512, 16, 40), f32)


def test_binding_refuses_matrices_it_cannot_pass():
    e4m3 = torch.float8_e4m3fn
    x, xs = torch.zeros(4, 256).to(e4m3), torch.zeros(4, 2)
    with pytest.raises(TypeError, match="dtype"):
        pkg.quantize_fp8(torch.zeros(4, 256, dtype=torch.float16))
    with pytest.raises(ValueError, match="GPU"):
        pkg.quantize_fp8(torch.zeros(4, 256))
    with pytest.raises(ValueError, match="dimensions"):
        pkg.quantize_fp8(torch.zeros(256))
    with pytest.raises(ValueError, match="contiguous"):
        pkg.quantize_fp8_weight(torch.zeros(256, 128).t())
    with pytest.raises(ValueError, match="GPU"):
        pkg.quantize_fp8_weight(torch.zeros(128))
    with pytest.raises(TypeError, match="dtype"):
        pkg.fp8_matmul(xs, xs, x, xs)
    with pytest.raises(ValueError, match="contiguous"):
        pkg.fp8_matmul(torch.zeros(256, 4).to(e4m3).t(), xs, x, xs)
    with pytest.raises(ValueError, match="GPU"):
        pkg.fp8_matmul(x, xs, x, xs)


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
