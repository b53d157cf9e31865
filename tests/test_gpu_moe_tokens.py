"""The sparse layer for a few tokens on the GPU against float64.

Bounds: logits are 64-bit sums rounded once, so the experts are those of the
oracle's fp32 logits.  Every product is exact or of three bf16 parts (24 bits)
and every sum fp32, so a sum of n terms is off by at most (n + 64) 2^-24 of the
sum of their magnitudes (n additions; parts, scales, the sums of eight waves and
the instruction's own additions, at most 2^-22 each, within the 64 where n is
small and within n where it is not); the oracle carries that through the
activation and the second product.  Then one rounding to the output's type."""

import numpy as np
import pytest
import torch

import sparse_moe_layer_latentmoe_amd as pkg
from oracle import operators as R

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F, B = torch.float32, torch.bfloat16
FORMATS = ["bf16", "fp8", "mxfp4"]


def rand(*shape, seed, dtype=F, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * std).to(dtype).to(DEV)


def quantised(w, fmt):
    """(codes, scales, float64 values) of weights [.., N, K]."""
    if fmt == "bf16":
        w = w.to(B)
        return w, None, w.double().cpu().numpy()
    if fmt == "fp8":
        c, s = pkg.quantize_fp8_weight(w)
        v = c.float().double() * s.double().repeat_interleave(128, -2).repeat_interleave(128, -1)
        return c, s, v.cpu().numpy()
    c, s = pkg.quantize_mxfp4(w.to(B))
    return c, s, R.dequantize_mxfp4(c.cpu().numpy(), s.cpu().numpy())


class Layer:
    def __init__(self, E, K, D, H, fmt="bf16", swiglu=False, S=0, seed=0, bias=True, gate_dtype=F,
                 **router):
        two = 2 if swiglu else 1
        self.router = pkg.make_router(E, K, **router)
        self.kw = dict(router)
        self.K, self.D, self.swiglu = K, D, swiglu
        self.gate = rand(E, D, seed=seed, std=D ** -0.5, dtype=gate_dtype)
        self.bias = rand(E, seed=seed + 1, std=0.1) if bias else None
        self.up = quantised(rand(E, two * H, D, seed=seed + 2, std=0.05), fmt)
        self.down = quantised(rand(E, D, H, seed=seed + 3, std=0.05), fmt)
        self.shared = None
        if S:
            self.shared = (quantised(rand(two * S, D, seed=seed + 4, std=0.05), fmt),
                           quantised(rand(D, S, seed=seed + 5, std=0.05), fmt))

    def __call__(self, x, out=B, stream=None):
        sh = {}
        if self.shared:
            (u, us, _), (d, ds, _) = self.shared
            sh = dict(shared_up=u, shared_down=d, shared_up_scales=us, shared_down_scales=ds)
        return pkg.moe_tokens(self.router, x, self.gate, self.up[0], self.down[0], bias=self.bias,
                              up_scales=self.up[1], down_scales=self.down[1],
                              activation=pkg.ACT_SWIGLU if self.swiglu else pkg.ACT_RELU2,
                              out_dtype=out, stream=stream, **sh)

    def check(self, x, out=B):
        y, idx, w = self(x, out)
        xd = x.double().cpu().numpy()
        logits = (xd @ self.gate.double().cpu().numpy().T).astype(np.float32).astype(np.float64)
        kw = dict(n_group=self.kw.get("n_group", 1), topk_group=self.kw.get("topk_group", 1),
                  softmax=self.kw.get("score") == pkg.SCORE_SOFTMAX,
                  renorm=self.kw.get("renormalise", True), scale=self.kw.get("scale", 1.0))
        bias = None if self.bias is None else self.bias.double().cpu().numpy()
        wi, ww = R.route(logits, bias, self.K, **kw)
        i = idx.cpu().numpy()
        assert np.array_equal(i, wi)
        # A score e^v or 1 / (1 + e^-v), v = l - max or l, in fp32: the difference
        # rounds by 2^-24 of itself, so do v log2 e and (by 2^-28) that constant,
        # which the exponential passes on as |v| (2^-24 + 2^-24 + 2^-28) of its
        # value; it, the sums, reciprocals and products add less than 2^-20.
        v = np.abs(logits) if not kw["softmax"] else logits.max(1, keepdims=True) - logits
        rel = 2.0 ** -20 + 1.1 * 2.0 ** -23 * v.max(1, keepdims=True)
        assert np.all(np.abs(w.double().cpu().numpy() - ww) <= rel * ww)
        sh = self.shared and (self.shared[0][2], self.shared[1][2])
        want, bound = R.moe_tokens(xd, i, w.double().cpu().numpy(), lambda e: self.up[2][e],
                                   lambda e: self.down[2][e], sh, self.swiglu)
        unit = torch.finfo(out).eps / 2
        err = np.abs(y.double().cpu().numpy() - want)
        # What lies below 2^-126 in fp32 (a square of 1e-32) may become 0: at most D
        # terms of each u, and H + S hidden values times weights below 1 for each
        # expert, fewer than 2^16 such losses in all.
        ok = bound * (1 + unit) + unit * np.abs(want) + 2.0 ** (16 - 126)
        assert y.dtype == out and np.all(err <= ok), float((err / np.maximum(ok, 1e-300)).max())
        return y


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("T,E,K,D,H,S", [
    (1, 8, 2, 128, 128, 0), (1, 1, 1, 128, 256, 128), (2, 60, 6, 256, 384, 128),
    (5, 16, 4, 640, 128, 0), (16, 8, 2, 384, 256, 256), (7, 130, 8, 256, 128, 0),
    (3, 520, 22, 256, 128, 0), (16, 4, 4, 1152, 640, 0), (16, 1, 1, 256, 2176, 0)])
def test_shapes(T, E, K, D, H, S, swiglu, fmt):
    layer = Layer(E, K, D, H, fmt, swiglu, S, seed=T + E, scale=2.5)
    layer.check(rand(T, D, seed=50 + T, dtype=B if T % 2 else F))
    layer.check(rand(T, D, seed=51 + T, dtype=F), out=F)


@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("D,H,S", [(64, 64, 0), (192, 704, 64), (1024, 320, 1408), (2112, 64, 0)])
def test_odd_widths_in_bf16(D, H, S, swiglu):
    for T in (1, 6, 16):
        layer = Layer(12, 3, D, H, "bf16", swiglu, S, seed=T, score=pkg.SCORE_SOFTMAX, bias=False)
        layer.check(rand(T, D, seed=T, dtype=B))


@pytest.mark.parametrize("fmt", FORMATS)
def test_wide(fmt):
    layer = Layer(6, 2, 2048, 5120, fmt, False, 0, seed=3)
    for T in (1, 16):
        layer.check(rand(T, 2048, seed=T), out=F)
    layer = Layer(2, 1, 8192, 256, fmt, True, 384, seed=3)
    layer.check(rand(11, 8192, seed=9, dtype=B))


@pytest.mark.parametrize("kw", [
    dict(score=pkg.SCORE_SOFTMAX, renormalise=False), dict(score=pkg.SCORE_SOFTMAX, scale=0.5),
    dict(n_group=8, topk_group=3, scale=5.0), dict(renormalise=False),
    dict(n_group=4, topk_group=1, group_score=2)])
@pytest.mark.parametrize("bias", [False, True])
def test_routers(kw, bias):
    layer = Layer(64, 6, 128, 64, bias=bias, seed=8, **kw)
    for T in (1, 9, 16):
        layer.check(rand(T, 128, seed=T, dtype=B))


def test_many_experts_and_bf16_router():
    for E in (129, 512, 1024):
        layer = Layer(E, 64, 64, 64, seed=E, gate_dtype=B)
        layer.check(rand(16, 64, seed=E, dtype=B), out=F)


@pytest.mark.parametrize("fmt", FORMATS)
def test_every_token_takes_the_same_experts(fmt):
    """16 rows an expert, wider than what fits at a time."""
    layer = Layer(32, 4, 1280, 896, fmt, seed=4)
    layer.bias = torch.zeros(32, device=DEV)
    layer.bias[[3, 9, 17, 31]] = 8.0
    layer.check(rand(16, 1280, seed=1), out=F)
    layer.check(rand(16, 1280, seed=2, dtype=B))


def test_values_of_very_different_size():
    layer = Layer(8, 2, 256, 256, seed=5)
    x = rand(4, 256, seed=6) * torch.exp(6 * rand(4, 256, seed=7))
    x[2] = 0.0
    x[3, :] = 0.0
    x[3, 17] = 1e-30
    layer.check(x, out=F)


def test_strided_rows_and_rows_behind_the_last():
    layer = Layer(16, 3, 256, 128, "mxfp4", S=128, seed=1)
    wide = rand(9, 800, seed=2, dtype=B)
    a = layer.check(wide[:5, 16:272])
    assert torch.equal(a, layer(wide[:5, 16:272].contiguous())[0])
    with pytest.raises(pkg.LmoeError):
        layer(wide[:, 1:257])           # not 16-byte aligned
    with pytest.raises(pkg.LmoeError):
        layer(rand(17, 256, seed=0))    # too many tokens


def test_no_tokens():
    y, idx, w = Layer(16, 3, 256, 128)(rand(0, 256, seed=0))
    assert y.shape == (0, 256) and idx.shape == (0, 3) and w.shape == (0, 3)


def test_workspace_in_any_state():
    layer = Layer(40, 5, 512, 256, "fp8", True, 128, seed=2)
    x = rand(8, 512, seed=3, dtype=B)
    want = layer(x)
    for fill in (0xFF, 0x7F, 0x01):
        torch.cuda.empty_cache()
        junk = [torch.full((1 << 22,), fill, dtype=torch.uint8, device=DEV) for _ in range(4)]
        torch.cuda.synchronize()
        del junk                          # the next call's workspace is cut from these
        assert all(torch.equal(a, b) for a, b in zip(layer(x), want))


@pytest.mark.parametrize("fmt", FORMATS)
def test_same_bits_on_streams_and_in_graphs(fmt):
    layer = Layer(48, 6, 512, 384, fmt, True, 256, seed=2)
    xs = [rand(6, 512, seed=s, dtype=B) for s in range(2)]
    want = [layer(x) for x in xs]
    sides = [torch.cuda.Stream() for _ in range(2)]
    for s in sides:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(20):                   # two at once
        got = [layer(x, stream=s) for x, s in zip(xs, sides)]
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert all(torch.equal(u, v) for u, v in zip(a, b))
    x = xs[0].clone()
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1):
        y1 = layer(x)
    with torch.cuda.graph(g2):
        y2 = layer(x)
    for seed in range(4):
        x.copy_(rand(6, 512, seed=20 + seed, dtype=B))
        g1.replay()
        g2.replay()
        torch.cuda.synchronize()
        want = layer(x)
        for a, b, c in zip(y1, want, y2):
            assert torch.equal(a, b) and torch.equal(c, b)


def test_agrees_with_routing_and_grouped_products():
    """The same layer from the calls that larger batches use: routing of the
    logits, 8-bit weights in grouped products; they quantise the activations,
    so the two agree to that (2^-4 of a value, about its root over many)."""
    T, E, K, D, H = 16, 24, 4, 512, 384
    layer = Layer(E, K, D, H, "fp8", seed=6, scale=2.0)
    x = rand(T, D, seed=7, dtype=B)
    y, idx, w = layer(x, out=F)
    logits = (x.double() @ layer.gate.double().t()).float()
    ridx, rw = pkg.route_logits(layer.router, logits, layer.bias)
    assert torch.equal(idx, ridx) and torch.equal(w, rw)
    order = idx.flatten().argsort(stable=True)
    off = torch.nn.functional.pad(torch.bincount(idx.flatten(), minlength=E).cumsum(0), (1, 0)).int()
    u = pkg.fp8_matmul(*pkg.quantize_fp8(x), *layer.up[:2], offsets=off, rows=(order // K).int(),
                       out_dtype=F)
    o = pkg.fp8_matmul(*pkg.quantize_fp8(torch.relu(u) ** 2), *layer.down[:2], offsets=off,
                       out_dtype=F)
    z = torch.zeros(T, D, device=DEV).index_add_(0, order // K, o * w.flatten()[order][:, None])
    assert float((z - y).norm() / y.norm()) < 2.0 ** -4


@pytest.mark.parametrize("out", [F, B])
def test_rows_that_are_not_finite_stay_alone(out):
    for T in (4, 11):                     # routed in the kernel and before it
        layer = Layer(40, 5, 256, 128, S=128, seed=3)
        x = rand(T, 256, seed=4)
        want = layer(x, out)
        x[1] = float("nan")
        x[3, 7] = float("inf")
        got = layer(x, out)
        keep = [t for t in range(T) if t not in (1, 3)]
        # a token's own sums are the same whoever shares its experts
        assert all(torch.equal(a[keep], b[keep]) for a, b in zip(got, want))
        assert bool(got[0][1].isnan().all()) and not bool(got[0][3].isfinite().any())
        i = got[1]
        assert bool((i >= 0).all()) and bool((i < 40).all()) and bool((i[:, 1:] > i[:, :-1]).all())


def test_values_next_to_the_largest():
    """x that rounds to infinity in bf16: its parts do not."""
    layer = Layer(8, 2, 128, 64, seed=3, swiglu=True, bias=False)
    big = torch.finfo(F).max
    layer.up = (layer.up[0] * 0, None, layer.up[2] * 0)
    layer.up[0][:, :64, 0] = layer.up[0][:, 64:, 1] = 2.0 ** -120
    layer.up[2][:, :64, 0] = layer.up[2][:, 64:, 1] = 2.0 ** -120
    x = torch.zeros(5, 128, device=DEV)
    x[:, 0], x[:, 1] = big, -big
    layer.gate = layer.gate * 2.0 ** -60
    layer.check(x, out=F)
    layer.check(x, out=B)


def test_a_bias_that_is_not_finite_stays_in_bounds():
    layer = Layer(200, 6, 128, 64, seed=3)
    x = rand(13, 128, seed=4)
    for bad in (float("nan"), float("inf"), -float("inf")):
        layer.bias = rand(200, seed=1)
        layer.bias[::3] = bad
        for T in (1, 4, 13):
            y, idx, w = layer(x[:T])
            assert bool((idx >= 0).all()) and bool((idx < 200).all())
    layer.bias = torch.full((200,), float("nan"), device=DEV)
    for T in (1, 4, 13):
        layer(x[:T])
    torch.cuda.synchronize()


def test_two_work_groups_a_cu():
    """Few tokens and much to read: 128 pairs of an expert of 5.5 MB."""
    layer = Layer(132, 32, 1024, 1344, seed=11, scale=2.0)
    layer.check(rand(4, 1024, seed=1), out=F)
    layer.check(rand(4, 1024, seed=2, dtype=B))
    layer = Layer(132, 32, 1024, 1408, "mxfp4", True, 128, seed=12)
    layer.check(rand(3, 1024, seed=3, dtype=B))


@pytest.mark.parametrize("D", [8192, 16384, 20480, 32768])
def test_one_token_of_a_wide_layer(D):
    """x in LDS before the first block, and where it does not fit."""
    for E, fmt in ((130, "bf16"), (6, "mxfp4")):
        layer = Layer(E, 3, D, 128, fmt, seed=D, S=128)
        layer.check(rand(1, D, seed=1), out=F)
        layer.check(rand(1, D, seed=2), out=B)
        layer.check(rand(1, D, seed=3, dtype=B))


def test_one_token_on_four_streams_at_once():
    """More work-groups of a CU's whole LDS than there are CUs: none waits for one
    that cannot start."""
    layer = Layer(160, 12, 1024, 1024, "fp8", S=1024, seed=2)
    xs = [rand(1, 1024, seed=s, dtype=B) for s in range(4)]
    want = [layer(x) for x in xs]
    sides = [torch.cuda.Stream() for _ in xs]
    for s in sides:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(20):
        got = [layer(x, stream=s) for x, s in zip(xs, sides)]
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert all(torch.equal(u, v) for u, v in zip(a, b))
