"""The layer with FP8 experts (expert_format = EXPERTS_FP8) and the operators
used together around it.

The layer is compared with the float64 oracle that quantises the same weights
and activations.  Routing does not depend on the format and must agree as for
bf16 experts.  The hidden rows are quantised after an fp32 sum on the GPU and
an fp64 sum in the oracle, so a value next to a rounding border may take the
neighbouring code: such a step is at most 2^-3 of one of F terms, the bf16
rounding of the expert outputs 2^-8; the layer's bar of 2e-2 normwise covers
both."""

import concurrent.futures

import numpy as np
import pytest
import torch

import lmoe_inputs as li
import sparse_moe_layer_latentmoe_amd as pkg
from oracle import lmoe_oracle as O
from oracle import operators as R
from parity import (MEDIUM, OUT_REL, TIE_GAP, check_properties, normwise_rel, oracle_config,
                    run_gpu, weight_dict)

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
SMALL = li.LayerShape(256, 128, 16, 4, 256, 512, 5.0)
WIDE = li.LayerShape(512, 384, 16, 4, 640, 512, 5.0)
MANY = li.LayerShape(512, 256, 64, 8, 384, 512, 5.0, 8, 4)


def fp8_weights(inp):
    w = weight_dict(inp)
    up, us = pkg.quantize_fp8_weight(inp.expert_up)
    dn, ds = pkg.quantize_fp8_weight(inp.expert_down)
    w.update(expert_up=None, expert_down=None, expert_up_fp8=up, expert_up_fp8_scale=us,
             expert_down_fp8=dn, expert_down_fp8_scale=ds)
    return w


class Coded:
    """obj[e]: expert e's weight as the oracle quantises it."""

    def __init__(self, bits):
        self.bits, self.made = bits, {}

    def __getitem__(self, e):
        if e not in self.made:
            self.made[e] = R.quantize_fp8(O.bf16_bits_to_f64(self.bits[e]).astype(np.float32), 128)
        return self.made[e]


def oracle(x, hw, cfg, up, down, idx):
    """(r, y) of the layer on x: bf16 bits, or float64 rows."""
    if x.dtype != np.float64:
        x = O.bf16_bits_to_f64(x)
    z32 = O.latent_projection(x, O.bf16_bits_to_f64(hw.fc1_latent)).astype(np.float32)
    _, s = O.router_scores(z32, hw.router)
    want, _, gap = O.select_experts(s, hw.router_bias, cfg.num_experts_per_tok, cfg.n_group,
                                    cfg.topk_group)
    assert np.array_equal(idx[gap >= TIE_GAP], want[gap >= TIE_GAP])
    w = O.renormalize(s, idx, cfg.routed_scaling_factor)
    r = R.experts_fp8(z32, idx, w, up, down)
    y = O.latent_up_projection(r, O.bf16_bits_to_f64(hw.fc2_latent))
    y += O.shared_expert(x, O.bf16_bits_to_f64(hw.shared_up), O.bf16_bits_to_f64(hw.shared_down))
    return r, y


@pytest.mark.parametrize("shape,tokens,path", [
    (SMALL, 1, pkg.PATH_AUTO), (SMALL, 5, pkg.PATH_AUTO), (SMALL, 37, pkg.PATH_AUTO),
    (SMALL, 64, pkg.PATH_STREAM), (WIDE, 33, pkg.PATH_STREAM), (WIDE, 200, pkg.PATH_AUTO),
    (MEDIUM, 3, pkg.PATH_AUTO), (MEDIUM, 150, pkg.PATH_AUTO), (MEDIUM, 400, pkg.PATH_AUTO),
    (MEDIUM, 900, pkg.PATH_AUTO), (MEDIUM, 64, pkg.PATH_TILED), (MANY, 77, pkg.PATH_AUTO),
    (MANY, 1000, pkg.PATH_AUTO)])
def test_layer_matches_oracle(shape, tokens, path):
    wl = li.Workload("fp8", shape, tokens)
    inp = li.make_inputs(wl, DEV)
    w = fp8_weights(inp)
    layer = pkg.LatentMoE(shape, w, tokens, path=path, expert_format=pkg.EXPERTS_FP8)
    g = run_gpu(layer, inp.x)
    check_properties(g, shape, tokens)
    hw = li.HostWeights(inp, eager_experts=True)
    up, down = Coded(hw.expert_up), Coded(hw.expert_down)
    r, y = oracle(li.bf16_bits(inp.x), hw, oracle_config(shape), up, down, g.idx)
    assert normwise_rel(g.r, r) <= OUT_REL
    assert normwise_rel(g.y.float().cpu().numpy(), y) <= OUT_REL
    for e in np.unique(g.idx)[:4]:
        assert np.array_equal(w["expert_up_fp8"][int(e)].view(torch.uint8).cpu().numpy(), up[e][0])
        assert np.array_equal(w["expert_down_fp8_scale"][int(e)].cpu().numpy(), down[e][1])
    # the allocation-free forward: the same bits
    if pkg.workspace_size(layer.cfg) <= pkg.NOALLOC_SCRATCH_BYTES:
        out = torch.full_like(inp.x, float("nan"))
        layer.forward_noalloc_into(inp.x, out)
        torch.cuda.synchronize()
        assert torch.equal(out.view(torch.int16), g.y.view(torch.int16))
    layer.close()


@pytest.fixture(scope="module")
def full():
    wl = li.workload("decode")
    weights = li.make_weights(wl, DEV)
    return weights, fp8_weights(li.make_inputs(wl, DEV, weights=weights))


@pytest.mark.fullshape
@pytest.mark.parametrize("name,tokens,rows", [("decode", None, [31]),
                                              ("mtp_verify", None, [100]),
                                              ("prefill", 21504, [0, 21503])])
def test_layer_at_full_shape(full, name, tokens, rows):
    """Streamed experts, 64-row tiles and the long batch on 192-row tiles (more
    than 2 GiB of hidden codes): properties on every token, and the whole
    output of a token or two against the oracle, which quantises the experts
    they use."""
    wl = li.workload(name) if tokens is None else li.workload(name, tokens=tokens)
    print(f"[fp8 full {name} T={wl.tokens}]", flush=True)
    weights, w = full
    inp = li.make_inputs(wl, DEV, weights=weights)
    layer = pkg.LatentMoE(wl.shape, w, wl.tokens, expert_format=pkg.EXPERTS_FP8)
    g = run_gpu(layer, inp.x)
    check_properties(g, wl.shape, wl.tokens)
    hw = li.HostWeights(inp)
    up, down = Coded(hw.expert_up), Coded(hw.expert_down)
    r, y = oracle(li.bf16_bits(inp.x[rows]), hw, oracle_config(wl.shape), up, down, g.idx[rows])
    assert normwise_rel(g.r[rows], r) <= OUT_REL
    assert normwise_rel(g.y[rows].float().cpu().numpy(), y) <= OUT_REL
    e = int(g.idx[rows[0], 0])
    assert np.array_equal(w["expert_up_fp8"][e].view(torch.uint8).cpu().numpy(), up[e][0])
    assert np.array_equal(w["expert_down_fp8_scale"][e].cpu().numpy(), down[e][1])
    layer.close()


def test_layer_refuses_widths_that_are_not_whole_blocks():
    sh = li.LayerShape(256, 192, 16, 4, 256, 512, 5.0)
    inp = li.make_inputs(li.Workload("fp8", sh, 4), DEV)
    with pytest.raises(pkg.LmoeError) as e:
        pkg.LatentMoE(sh, fp8_weights(inp), 4, expert_format=pkg.EXPERTS_FP8)
    assert e.value.status == pkg.LMOE_ERR_UNSUPPORTED
    w = weight_dict(li.make_inputs(li.Workload("fp8", SMALL, 4), DEV))
    with pytest.raises(ValueError, match="expert_up_fp8"):
        pkg.LatentMoE(SMALL, w, 4, expert_format=pkg.EXPERTS_FP8)


def test_layer_with_fewer_tokens_than_it_was_made_for():
    inp = li.make_inputs(li.Workload("fp8", MEDIUM, 900), DEV)
    w = fp8_weights(inp)
    large = pkg.LatentMoE(MEDIUM, w, 900, expert_format=pkg.EXPERTS_FP8)
    for T in (900, 1, 150, 400, 37):
        one = pkg.LatentMoE(MEDIUM, w, T, expert_format=pkg.EXPERTS_FP8)
        assert torch.equal(large.forward(inp.x[:T]), one.forward(inp.x[:T]))
        one.close()
    large.close()


@pytest.mark.parametrize("tokens", [5, 300])
def test_layer_inside_its_block(tokens):
    """The fused pre-norm and residual around FP8 experts: their epilogues hand
    the quantiser the normalised latent."""
    wl = li.Workload("fp8", SMALL, tokens)
    inp = li.make_inputs(wl, DEV)
    gamma = li.make_norm_weight(wl, DEV)
    w = dict(fp8_weights(inp), norm_weight=gamma)
    layer = pkg.LatentMoE(SMALL, w, tokens, expert_format=pkg.EXPERTS_FP8, fuse=pkg.FUSE_BLOCK)
    g = run_gpu(layer, inp.x)
    hw = li.HostWeights(inp, eager_experts=True)
    h = li.bf16_bits(inp.x)
    xt, rn = O.rms_prenorm(h, li.bf16_bits(gamma))
    r, y = oracle(rn[:, None] * O.bf16_bits_to_f64(xt), hw, oracle_config(SMALL),
                  Coded(hw.expert_up), Coded(hw.expert_down), g.idx)
    assert normwise_rel(g.r, r) <= OUT_REL
    assert normwise_rel(g.y.float().cpu().numpy(), O.bf16_bits_to_f64(h) + y) <= OUT_REL
    layer.close()


def test_operators_on_two_streams_at_once():
    """Calls that run at the same time share nothing: the bits of calls made alone."""
    g = torch.Generator().manual_seed(3)
    rnd = lambda *n: torch.randn(*n, generator=g).to(DEV)  # noqa: E731
    wc, ws = pkg.quantize_fp8_weight(rnd(6, 512, 1024) * 0.02)
    dc, ds = pkg.quantize_fp8_weight(rnd(256, 1024) * 0.02)
    post, gate = rnd(1024), rnd(1024)
    router = pkg.make_router(64, 8, n_group=8, topk_group=4)

    def work(x, y, stream):
        c, sc = pkg.quantize_fp8(x, stream=stream)
        off = torch.tensor([0, 7, 7, 90, 91, 250, x.shape[0]], dtype=torch.int32).to(DEV)
        torch.cuda.synchronize()
        out = []
        for _ in range(8):
            h, n, st = pkg.block_norm(x, y, pre_weight=gate, post_weight=post, gate=gate,
                                      want_stats=True, stream=stream)
            gr = pkg.block_norm_backward(x, y, st, dh_out=x, dx=y, pre_weight=gate,
                                         post_weight=post, gate=gate, stream=stream)
            out.append([pkg.fp8_matmul(c, sc, wc, ws, off, stream=stream),      # tile list
                        pkg.fp8_matmul(c, sc, dc, ds, stream=stream),           # parts of k
                        *pkg.route_logits(router, x[:, :64], stream=stream),
                        h, n, gr.dh, gr.dy, gr.dpre_weight, gr.dpost_weight, gr.dgate])
        return out

    xs, ys = [rnd(400, 1024) for _ in range(2)], [rnd(400, 1024) for _ in range(2)]
    want = [work(x, y, None)[0] for x, y in zip(xs, ys)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    with concurrent.futures.ThreadPoolExecutor(2) as pool:
        got = list(pool.map(work, xs, ys, streams))
    torch.cuda.synchronize()
    for runs, alone in zip(got, want):
        for r in runs:
            assert all(torch.equal(a, b) for a, b in zip(r, alone))


def test_layer_replays_from_a_graph():
    T = 48
    inp = li.make_inputs(li.Workload("fp8", MEDIUM, T), DEV)
    layer = pkg.LatentMoE(MEDIUM, fp8_weights(inp), T, expert_format=pkg.EXPERTS_FP8)
    x = inp.x.clone()
    y = torch.empty_like(x)
    layer.forward_into(x, y)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        layer.forward_into(x, y)
    for seed in range(3):
        x.copy_(torch.randn(x.shape, generator=torch.Generator().manual_seed(seed)))
        g.replay()
        torch.cuda.synchronize()
        got = y.clone()
        layer.forward_into(x, y)
        torch.cuda.synchronize()
        assert torch.equal(got, y)
    layer.close()


def test_operators_as_one_block():
    """A block as a caller runs it: pre-norm, the layer with FP8 experts, the
    norms and gate behind it; and the layer's routed part rebuilt from the
    operators alone, which must give what the layer computes."""
    sh, T = MEDIUM, 96
    D, E, K = sh.hidden_size, sh.n_routed_experts, sh.num_experts_per_tok
    inp = li.make_inputs(li.Workload("fp8", sh, T), DEV)
    w = fp8_weights(inp)
    layer = pkg.LatentMoE(sh, w, T, expert_format=pkg.EXPERTS_FP8)
    ones = torch.ones(D, device=DEV)
    pre, post, gate = (ones + 0.1 * torch.randn(D, generator=torch.Generator().manual_seed(i)).to(DEV)
                       for i in range(3))
    h = inp.x.float() * 2
    _, x, _ = pkg.block_norm(h, None, pre_weight=pre)
    taps = pkg.Taps(z_f32=torch.empty(T, sh.moe_latent_size, device=DEV),
                    topk_idx=torch.empty(T, K, dtype=torch.int32, device=DEV),
                    topk_w=torch.empty(T, K, device=DEV),
                    r_latent=torch.empty(T, sh.moe_latent_size, device=DEV))
    y = layer.forward(x, taps)
    h2, x2, _ = pkg.block_norm(h, y, pre_weight=pre, post_weight=post, gate=gate)
    e64 = lambda t: t.double().cpu().numpy()  # noqa: E731
    want = R.block_norm(e64(h), None, e64(pre), None, None, None, 1e-5)[1]
    assert np.abs(e64(x) - want).max() <= 2.0 ** -7 * np.abs(want).max()
    w2 = R.block_norm(e64(h), e64(y), e64(pre), e64(post), e64(gate), None, 1e-5)
    assert np.abs(e64(h2) - w2[0]).max() <= 2.0 ** -17 * np.abs(w2[0]).max()
    assert np.abs(e64(x2) - w2[1]).max() <= 2.0 ** -7 * np.abs(w2[1]).max()
    # the routed experts, step by step
    logits = taps.z_f32 @ w["router"].t()
    r = pkg.make_router(E, K, scale=sh.routed_scaling_factor)
    idx, tw = pkg.route_logits(r, logits, w["router_bias"])
    assert torch.equal(idx, taps.topk_idx)
    # the layer's logits and these differ by their sums' rounding
    assert (tw - taps.topk_w).abs().max() <= 1e-4
    order = torch.sort(idx.reshape(-1).long(), stable=True).indices
    counts = torch.bincount(idx.reshape(-1).long(), minlength=E)
    off = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).int()
    zc, zs = pkg.quantize_fp8(taps.z_f32)
    u = pkg.fp8_matmul(zc, zs, w["expert_up_fp8"], w["expert_up_fp8_scale"], off,
                       (order // K).int(), out_dtype=torch.float32)
    hc, hs = pkg.quantize_fp8(torch.relu(u) ** 2)
    o = pkg.fp8_matmul(hc, hs, w["expert_down_fp8"], w["expert_down_fp8_scale"], off)
    slots = torch.empty_like(o)
    slots[order] = o
    rr = (slots.view(T, K, -1).float() * tw[:, :, None]).sum(1)
    # The layer quantises its hidden rows from sums that keep about 17 bits, u
    # here is fp32: they differ by up to 2^-15.9 of u's terms' magnitudes, whose
    # sum is 2/pi sqrt(256) = 10.2 times u's root mean square.  So h = u^2 and the
    # scale of its block may each be off by 2 * 10.2 * 2^-15.9 = 2^-11.5 of h, and
    # with codes at least 2^-4 apart a fraction of 2 * 2^-11.5 / 2^-4 = 2^-6.5 of
    # them may be neighbours, at most 2^-3 away: sqrt(2^-6.5) 2^-3 = 1.3e-2 of
    # the values (root mean squares; the largest error and the largest value of
    # as many sums stand in the same ratio), and 2^-8 for the bf16 rows.
    assert normwise_rel(rr.cpu().numpy(), e64(taps.r_latent)) <= 1.3e-2 + 2.0 ** -8
    layer.close()
