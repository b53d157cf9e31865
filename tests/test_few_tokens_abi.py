"""4-bit activations and products and the layer for a few tokens on the CPU: the
C ABI refuses bad arguments before any HIP call, the binding refuses tensors
that the kernels could not take, and the oracle agrees with itself."""

import numpy as np
import pytest
import torch

import sparse_moe_layer_latentmoe_amd as pkg
from oracle import operators as R

FAKE = 0x10000000     # never dereferenced
INV, UNS, WS = pkg.LMOE_ERR_INVALID_ARG, pkg.LMOE_ERR_UNSUPPORTED, pkg.LMOE_ERR_WORKSPACE
U8, F, B = torch.uint8, torch.float32, torch.bfloat16


@pytest.fixture(scope="module")
def lib():
    return pkg.load_library()


def at(i):
    return FAKE + (i << 36)


def fill(a, base, kw):
    for k, v in {**base, **kw}.items():
        setattr(a, k, v)
    return a


# ---- quantiser and the way back ----------------------------------------------


def test_quantiser_arguments_are_checked(lib):
    base = dict(x=at(0), t=1, rows=4, cols=200, stride=200, codes=at(1), scales=at(2))

    def call(**kw):
        v = {**base, **kw}
        return lib.lmoe_quantize_mxfp4_rows(v["x"], v["t"], v["rows"], v["cols"], v["stride"],
                                            v["codes"], v["scales"], None)

    assert call(rows=0, x=None, codes=None, scales=None) == pkg.LMOE_OK
    # 7 blocks a row: 448 bytes of codes, 28 scales
    for kw in (dict(x=None), dict(codes=None), dict(scales=None), dict(t=2), dict(t=-1),
               dict(rows=-1), dict(cols=0), dict(cols=-3), dict(stride=199), dict(x=at(0) + 1),
               dict(codes=at(1) + 2), dict(codes=at(0) + 1596), dict(scales=at(1) + 447),
               dict(t=0, x=at(0) + 2), dict(codes=at(2) + 24), dict(scales=at(0))):
        assert call(**kw) == INV, kw
    assert call(rows=1 << 28) == UNS                   # 7 2^28 blocks
    assert call(rows=(1 << 30) - 63, cols=1, stride=1) == UNS
    assert call(rows=1 << 41, cols=1, stride=1) == UNS
    assert call(rows=1, cols=(1 << 30) + 1, stride=1 << 31) == UNS
    assert call(stride=(1 << 31) + 1) == UNS


def test_way_back_arguments_are_checked(lib):
    base = dict(codes=at(0), scales=at(1), rows=4, cols=200, y=at(2), t=1)

    def call(**kw):
        v = {**base, **kw}
        return lib.lmoe_dequantize_mxfp4(v["codes"], v["scales"], v["rows"], v["cols"], v["y"],
                                         v["t"], None)

    assert call(rows=0, codes=None, scales=None, y=None) == pkg.LMOE_OK
    for kw in (dict(codes=None), dict(scales=None), dict(y=None), dict(t=2), dict(rows=-1),
               dict(cols=0), dict(codes=at(0) + 1), dict(y=at(2) + 1), dict(t=0, y=at(2) + 2),
               dict(y=at(0) + 444), dict(y=at(1) + 24), dict(y=at(1) - 1596)):
        assert call(**kw) == INV, kw
    assert call(rows=1 << 28) == UNS
    assert call(rows=1, cols=(1 << 30) + 1) == UNS


# ---- products -----------------------------------------------------------------


def mm_args(**kw):
    return fill(pkg.LmoeMxfp4MatmulArgs(), dict(
        x=at(0), x_scales=at(1), w=at(2), w_scales=at(3), rows=None, offsets=None, y=at(4),
        y_type=1, n_groups=0, M=40, x_rows=40, N=256, K=1024), kw)


@pytest.mark.parametrize("kw,status", [
    (dict(M=-1), INV), (dict(N=0), INV), (dict(K=0), INV), (dict(n_groups=-1), INV),
    (dict(x_rows=0), INV), (dict(y_type=2), INV), (dict(x=None), INV), (dict(x_scales=None), INV),
    (dict(w=None), INV), (dict(w_scales=None), INV), (dict(y=None), INV),
    (dict(x=at(0) + 8), INV), (dict(w=at(2) + 4), INV), (dict(y=at(4) + 8), INV),
    (dict(w_scales=at(3) + 2), INV), (dict(x_scales=at(1) + 1), INV), (dict(rows=at(5) + 2), INV),
    (dict(x_rows=39), INV), (dict(offsets=at(5)), INV), (dict(n_groups=3), INV),
    (dict(N=250), UNS), (dict(K=1056), UNS), (dict(K=65664), UNS), (dict(N=(1 << 20) + 16), UNS),
    (dict(M=(1 << 24) + 1, x_rows=1 << 25), UNS), (dict(n_groups=1025, offsets=at(5)), UNS),
    (dict(rows=at(5), x_rows=1 << 22), UNS)])
def test_product_arguments_are_checked(lib, kw, status):
    a = mm_args(**kw)
    assert lib.lmoe_mxfp4_matmul_workspace_size(a) == 0
    assert lib.lmoe_mxfp4_matmul(a, at(6), 1 << 30, None) == status


@pytest.mark.parametrize("kw", [
    dict(y=at(0) + 1024), dict(y=at(2) + (1 << 17) - 16), dict(y=at(1) - 16), dict(y=at(3)),
    dict(rows=at(4) + 32), dict(n_groups=3, offsets=at(4))])
def test_products_do_not_overwrite_what_they_read(lib, kw):
    assert lib.lmoe_mxfp4_matmul(mm_args(**kw), at(6), 1 << 30, None) == INV


def test_product_workspace_is_checked(lib):
    size, mm = lib.lmoe_mxfp4_matmul_workspace_size, lib.lmoe_mxfp4_matmul
    assert mm(None, None, 0, None) == INV and size(None) == 0
    assert size(mm_args(M=0)) == 0 and mm(mm_args(M=0, x=None), None, 0, None) == pkg.LMOE_OK
    assert size(mm_args(M=5)) == 0                     # one pass over the weights
    split = mm_args(M=150, x_rows=150, N=512, K=16384)  # few tiles: k is split
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
    assert size(split) % (150 * 512 * 4) == 0


# ---- the layer for a few tokens ------------------------------------------------


def few_args(router=None, **kw):
    """T 4 of 16 experts top-4, D 256, F 384, S 128 in MXFP4."""
    return fill(pkg.LmoeMoeTokensArgs(), dict(
        router=pkg.make_router(16, 4) if router is None else router, x=at(0), x_stride=256,
        gate=at(1), bias=at(2), up=at(3), down=at(4), shared_up=at(5), shared_down=at(6),
        up_scales=at(7), down_scales=at(8), shared_up_scales=at(9), shared_down_scales=at(10),
        y=at(11), topk_idx=at(12), topk_w=at(13), x_type=1, gate_type=0, y_type=1,
        expert_format=pkg.EXPERTS_MXFP4, activation=pkg.ACT_RELU2, T=4, D=256, F=384, S=128), kw)


NO_SHARED = dict(S=0, shared_up=None, shared_down=None, shared_up_scales=None,
                 shared_down_scales=None)
PLAIN = dict(expert_format=pkg.EXPERTS_BF16, up_scales=None, down_scales=None,
             shared_up_scales=None, shared_down_scales=None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), INV), (dict(T=17), pkg.LMOE_ERR_TOO_MANY_TOKENS), (dict(D=0), INV),
    (dict(F=-128), INV), (dict(F=0), INV), (dict(S=-128), INV), (dict(x_type=2), INV),
    (dict(gate_type=-1), INV), (dict(y_type=7), INV), (dict(expert_format=3), INV),
    (dict(expert_format=-1), INV), (dict(activation=2), INV), (dict(D=192, x_stride=192), UNS),
    (dict(F=448), UNS), (dict(S=64), UNS), (dict(F=32896), UNS), (dict(D=32896), UNS),
    (dict(D=96, **PLAIN), UNS),
    # 2^31 bytes a matrix
    (dict(D=32768, F=32768, **PLAIN), UNS), (dict(S=32768, D=32768, F=64, **PLAIN), UNS),
    (dict(D=32768, F=32768, activation=1, expert_format=2), UNS),
    (dict(router=pkg.make_router(1025, 4)), UNS), (dict(router=pkg.make_router(256, 65)), UNS),
    (dict(router=pkg.make_router(16, 17)), INV), (dict(router=pkg.make_router(16, 0)), INV),
    (dict(router=pkg.make_router(16, 4, scale=float("inf"))), INV)])
def test_few_token_settings_are_checked(lib, kw, status):
    a = few_args(**kw)
    assert lib.lmoe_moe_tokens_workspace_size(a) == 0
    assert lib.lmoe_moe_tokens(a, at(14), 1 << 40, None) == status


POINTERS = ("x", "gate", "up", "down", "shared_up", "shared_down", "up_scales", "down_scales",
            "shared_up_scales", "shared_down_scales", "y")


@pytest.mark.parametrize("kw", [
    *({n: None} for n in POINTERS + ("topk_idx", "topk_w")),
    *({n: at(15) + 8} for n in POINTERS),
    dict(bias=at(2) + 2), dict(topk_idx=at(12) + 1), dict(topk_w=at(13) + 2), dict(x_stride=248),
    dict(x_stride=260), {**NO_SHARED, "shared_up": at(5)}, {**NO_SHARED, "shared_down": at(6)},
    {**NO_SHARED, "shared_up_scales": at(9)}, dict(S=0), {**PLAIN, "up_scales": at(7)},
    {**PLAIN, "shared_down_scales": at(7)}, dict(expert_format=pkg.EXPERTS_BF16),
    # outputs on inputs and on each other
    *({"y": at(i) + 16} for i in (0, 1, 3, 4, 5, 6, 7, 8, 9, 10)), dict(y=at(2) - 16),
    dict(topk_idx=at(11) + 4), dict(topk_w=at(12)), dict(topk_w=at(2) + 60),
    dict(topk_idx=at(3) + 16 * 384 * 128 - 4)])
def test_few_token_arguments_are_checked(lib, kw):
    a = few_args(**kw)
    assert lib.lmoe_moe_tokens(a, at(14), 1 << 40, None) == INV


def test_few_token_workspace_is_checked(lib):
    size, run = lib.lmoe_moe_tokens_workspace_size, lib.lmoe_moe_tokens
    assert run(None, None, 0, None) == INV and size(None) == 0
    assert size(few_args(T=0)) == 0
    assert run(few_args(T=0, x=None, y=None), None, 0, None) == pkg.LMOE_OK
    for a in (few_args(), few_args(**NO_SHARED), few_args(activation=1), few_args(T=16, **PLAIN)):
        need = size(a)
        # logits, hidden rows, output rows
        assert need >= 4 * a.T * (16 + 4 * a.F + a.S + (4 + (a.S > 0)) * a.D)
        assert run(a, None, need, None) == WS
        assert run(a, at(14), need - 1, None) == WS
        assert run(a, at(14) + 128, need, None) == WS
        for i in (0, 1, 3, 4, 11, 12):
            assert run(a, at(i), need, None) == INV, i
    assert run(few_args(x_stride=(1 << 31) + 8), at(14), 1 << 40, None) == UNS
    # one token more is never less; nothing depends on pointers
    sizes = [size(few_args(T=t, x=None)) for t in range(17)]
    assert sizes == sorted(sizes) and sizes[16] < 1 << 20


# ---- the binding ---------------------------------------------------------------


def test_binding_refuses_matrices_it_cannot_pass():
    q, d, mm = pkg.quantize_mxfp4_rows, pkg.dequantize_mxfp4, pkg.mxfp4_matmul
    x, xs = torch.zeros(4, 128, dtype=U8), torch.zeros(4, 8, dtype=U8)
    for call, kind, match in (
            (lambda: q(torch.zeros(4, 256, dtype=torch.float16)), TypeError, "dtype"),
            (lambda: q(torch.zeros(256)), ValueError, "dimensions"),
            (lambda: q(torch.zeros(4, 256).t()), ValueError, "rows"),
            (lambda: q(torch.zeros(4, 256)), ValueError, "GPU"),
            (lambda: q(torch.zeros(4, 256, requires_grad=True)), (ValueError, RuntimeError), "grad"),
            (lambda: d(x.float(), xs), (TypeError, ValueError), "scales|codes"),
            (lambda: d(x, xs), ValueError, "GPU"),
            (lambda: mm(x.float(), xs, x, xs), TypeError, "dtype"),
            (lambda: mm(torch.zeros(128, 4, dtype=U8).t(), xs, x, xs), ValueError, "contiguous"),
            (lambda: mm(x, xs, x, xs), ValueError, "GPU")):
        with pytest.raises(kind, match=match):
            call()


def test_binding_refuses_layers_it_cannot_pass():
    r = pkg.make_router(16, 4)
    x = torch.zeros(2, 128)
    gate, up, down = torch.zeros(16, 128), torch.zeros(16, 64, 128), torch.zeros(16, 128, 64)
    with pytest.raises((ValueError, RuntimeError), match="grad"):
        pkg.moe_tokens(r, x.requires_grad_(), gate, up, down)
    with pytest.raises((ValueError, RuntimeError), match="grad"):
        pkg.moe_tokens(r, x.detach(), gate, up, down.requires_grad_())
    x, down = x.detach(), down.detach()
    with pytest.raises(TypeError, match="dtype"):
        pkg.moe_tokens(r, x.half(), gate, up, down)
    with pytest.raises(ValueError, match="dimensions"):
        pkg.moe_tokens(r, x[0], gate, up, down)
    with pytest.raises(ValueError, match="GPU"):
        pkg.moe_tokens(r, x, gate, up, down)


# ---- the oracle ----------------------------------------------------------------


def test_oracle_quantises_to_the_nearest():
    """No other code of the same scale is nearer, and values that are already of
    the grid come back as they are."""
    g = np.random.default_rng(3)
    x = g.normal(size=(5, 70)) * np.exp(g.normal(size=(5, 1)) * 4)
    c, s = R.quantize_mxfp4_rows(x)
    v = R.dequantize_mxfp4(c, s)
    assert v.shape == (5, 96) and not v[:, 70:].any()
    grid = np.concatenate([R.E2M1, -R.E2M1])
    step = np.ldexp(1.0, s.astype(int) - 127).repeat(32, 1)[:, :70]
    best = np.abs(x[..., None] - grid * step[..., None]).min(-1)
    assert np.array_equal(np.abs(x - v[:, :70]), best)
    c2, s2 = R.quantize_mxfp4_rows(v)
    assert np.array_equal(R.dequantize_mxfp4(c2, s2), v)


@pytest.mark.parametrize("swiglu", [False, True])
def test_oracle_layer_is_the_sum_over_pairs(swiglu):
    g = np.random.default_rng(4)
    T, E, K, D, H = 5, 7, 3, 12, 10
    two = 2 if swiglu else 1
    x, up, down = g.normal(size=(T, D)), g.normal(size=(E, two * H, D)), g.normal(size=(E, D, H))
    sh = (g.normal(size=(two * H, D)), g.normal(size=(D, H)))
    idx, w = R.route(g.normal(size=(T, E)), None, K, scale=1.5)

    def expert(v, u, d):
        a = u @ v
        return d @ (a[:H] / (1 + np.exp(-a[:H])) * a[H:] if swiglu else np.maximum(a, 0) ** 2)

    want = np.stack([sum(w[t, k] * expert(x[t], up[idx[t, k]], down[idx[t, k]]) for k in range(K))
                     + expert(x[t], *sh) for t in range(T)])
    y, bound = R.moe_tokens(x, idx, w, lambda e: up[e], lambda e: down[e], sh, swiglu)
    # float64 against float64: a few hundred roundings of 2^-53
    assert np.allclose(y, want, rtol=1e-12, atol=1e-10)
    # the bound, of 2^-24 roundings, is not below float64's and far below the values
    assert np.all(bound > 0) and bound.max() < 1e-3 * np.abs(want).max()
