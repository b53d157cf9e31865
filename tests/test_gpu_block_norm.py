"""The norms around a block on the GPU against the float64 oracle.

Bounds.  A row's sum of squares is a chain of at most 16 fused additions a
thread, six butterfly steps and 16 additions of wave sums: 38 half-ulps,
halved by the root, plus division and root: ry and rh within 2^-19.  h_out
adds a product chain: 2^-18 of |res_scale h| + |gate n|; x multiplies by rh
and pre: 2^-17.  Gradients chain two such rows' sums and differences whose
terms' magnitudes the oracle adds up: 2^-15 of that (column sums add at most
T / work-groups + 24 more half-ulps of it).  Each result then rounds once to
its type: half an ulp, 2^-8 for bf16."""

import numpy as np
import pytest
import torch

import sparse_moe_layer_latentmoe_amd as pkg
from oracle import operators as R

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F, B = torch.float32, torch.bfloat16


def exact(t):
    return None if t is None else t.double().cpu().numpy()


def rand(*shape, seed, dtype=F, std=1.0, mean=0.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * std + mean).to(dtype).to(DEV)


def unit(t):
    return torch.finfo(t.dtype).eps / 2


def close(got, want, mag, rel, what):
    err = np.abs(exact(got) - want)
    ok = rel * mag + unit(got) * (np.abs(want) + rel * mag) + 1e-37
    assert np.all(err <= ok), (what, float((err / ok).max()))


def check(T, D, ht=B, yt=B, pt=B, gate="channel", post=True, pre=True, alpha=True, y=True,
          pad=0, seed=0, train=True, eps=1e-5, zero_rows=()):
    h = rand(T, D + pad, seed=seed, dtype=ht, std=3.0)[:, pad // 2:pad // 2 + D]
    yv = rand(T, D + pad, seed=seed + 1, dtype=yt)[:, pad // 2:pad // 2 + D] if y else None
    for r in zero_rows:
        h[r] = 0
        if y:
            yv[r] = 0
    p = dict(pre_weight=rand(D, seed=seed + 2, dtype=pt, std=0.1, mean=1.0) if pre else None,
             post_weight=rand(D, seed=seed + 3, dtype=pt, std=0.1, mean=1.0) if post else None,
             res_scale=rand(D, seed=seed + 4, dtype=pt, std=0.1, mean=1.0) if alpha else None,
             gate={"none": lambda: None, "channel": lambda: rand(D, seed=seed + 5, dtype=pt),
                   "token": lambda: rand(T, 1, seed=seed + 5, dtype=pt),
                   "full": lambda: rand(T, D, seed=seed + 5, dtype=pt)}[gate]())
    h2, x, stats = pkg.block_norm(h, yv, eps=eps, want_stats=True, **p)
    e = {k: exact(v) for k, v in p.items()}
    want = R.block_norm(exact(h), exact(yv), e["pre_weight"], e["post_weight"], e["gate"],
                        e["res_scale"], eps)
    ab = lambda v: None if v is None else np.abs(v)  # noqa: E731
    a1 = 1.0 if e["res_scale"] is None else e["res_scale"]
    g1 = 1.0 if e["gate"] is None else e["gate"]
    n = np.zeros((T, D)) if not y else exact(yv) * want[2] * (e["post_weight"] if post else 1.0)
    mag = np.abs(a1 * exact(h)) + np.abs(g1 * n)
    close(h2, want[0], mag, 2.0 ** -18, "h_out")
    assert h2.dtype == ht
    if pre:
        close(x, want[1], np.abs(e["pre_weight"]) * mag * want[3], 2.0 ** -17, "x")
        assert x.dtype == (yt if y else B)
    else:
        assert x is None
    assert np.allclose(exact(stats), np.concatenate(want[2:], 1), rtol=2.0 ** -18, atol=0)
    if not train:
        return
    dh = rand(T, D, seed=seed + 6, dtype=ht)
    dx = rand(T, D, seed=seed + 7, dtype=yt if y else B) if pre else None
    g = pkg.block_norm_backward(h, yv, stats, dh_out=dh, dx=dx, eps=eps, **p)
    back = R.block_norm_backward(exact(h), exact(yv), exact(dh), exact(dx), e["pre_weight"],
                                 e["post_weight"], e["gate"], e["res_scale"], eps)
    for name in ("dh", "dy", "dpre_weight", "dpost_weight", "dres_scale", "dgate"):
        got = getattr(g, name)
        assert (got is None) == (name not in back), name
        if got is not None:
            close(got, *back[name], 2.0 ** -15, name)
    # either upstream gradient alone
    g1 = pkg.block_norm_backward(h, yv, stats, dh_out=dh, eps=eps, **p)
    b1 = R.block_norm_backward(exact(h), exact(yv), exact(dh), None, e["pre_weight"],
                               e["post_weight"], e["gate"], e["res_scale"], eps)
    close(g1.dh, *b1["dh"], 2.0 ** -15, "dh alone")
    if pre:
        assert not g1.dpre_weight.any()
        g2 = pkg.block_norm_backward(h, yv, stats, dx=dx, eps=eps, **p)
        b2 = R.block_norm_backward(exact(h), exact(yv), None, exact(dx), e["pre_weight"],
                                   e["post_weight"], e["gate"], e["res_scale"], eps)
        for name in ("dh", "dy", "dpre_weight", "dgate"):
            if name in b2:
                close(getattr(g2, name), *b2[name], 2.0 ** -15, name + " of x alone")


@pytest.mark.parametrize("T", [1, 5, 67])
@pytest.mark.parametrize("D", [1, 3, 8, 64, 100, 512, 520, 1000, 2048, 2056, 4096, 8192, 8191])
def test_widths(T, D):
    check(T, D, seed=T + D)


@pytest.mark.parametrize("D", [8200, 10240, 16384, 12001])
def test_rows_wider_than_the_layer(D):
    check(3, D, ht=F)


@pytest.mark.parametrize("gate", ["none", "channel", "token", "full"])
@pytest.mark.parametrize("ht,yt,pt", [(B, B, F), (F, B, B), (F, F, F), (B, F, B)])
def test_types_and_gates(gate, ht, yt, pt):
    check(37, 768, ht, yt, pt, gate)
    check(9, 333, ht, yt, pt, gate)


@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("pre", [True, False])
@pytest.mark.parametrize("alpha", [True, False])
def test_parts_left_out(post, pre, alpha):
    for gate in ("none", "channel", "token", "full"):
        check(11, 256, post=post, pre=pre, alpha=alpha, gate=gate)
    check(11, 256, post=False, pre=pre, alpha=alpha, gate="none", y=False)


@pytest.mark.parametrize("D,pad", [(256, 8), (256, 64), (256, 3), (1024, 2), (4096, 8)])
def test_strided_rows(D, pad):
    check(21, D, pad=pad)
    check(21, D, pad=pad, ht=F, gate="full")


def test_many_rows_column_sums():
    check(4099, 512, gate="channel")
    check(3001, 136, ht=F, yt=F, pt=F, gate="token")


def test_rows_of_zeros():
    check(6, 512, zero_rows=(0, 3), eps=1e-6)


def test_no_rows_and_untouched_rows():
    D = 256
    w = rand(D, seed=1, dtype=B)
    h = rand(0, D, seed=0, dtype=B)
    h2, x, st = pkg.block_norm(h, h, pre_weight=w, post_weight=w, gate=w, want_stats=True)
    assert h2.shape == x.shape == (0, D) and st.shape == (0, 2)
    g = pkg.block_norm_backward(h, h, st, dh_out=h2, dx=x, pre_weight=w, post_weight=w, gate=w)
    for t in (g.dpre_weight, g.dpost_weight, g.dgate):
        assert t.shape == (D,) and not t.any()
    # the C ABI on the first rows of longer arrays leaves the rest alone
    lib = pkg.load_library()
    full = torch.full((8, D), 7.0, dtype=B, device=DEV)
    xo = full.clone()
    src = rand(8, D, seed=4, dtype=B)
    a = pkg.LmoeBlockNormArgs(h=src.data_ptr(), h_stride=D, h_type=1, y_type=1, T=5, D=D, eps=1e-5)
    assert lib.lmoe_block_norm(a, full.data_ptr(), xo.data_ptr(), None,
                               torch.cuda.current_stream().cuda_stream) == 0
    torch.cuda.synchronize()
    assert torch.equal(full[:5], src[:5]) and bool((full[5:] == 7).all() & (xo[5:] == 7).all())


def test_rows_further_apart_than_32_bits():
    D = 64
    h, y, dh, dx = (rand(2, D, seed=5 + i, dtype=B) for i in range(4))
    far = [torch.empty(2, 2 ** 31, dtype=B, device=DEV)[:, :D] for _ in range(2)]
    for f, v in zip(far, (h, y)):
        f.copy_(v)
    par = dict(pre_weight=rand(D, seed=1), post_weight=rand(D, seed=2), gate=rand(2, D, seed=3))
    out = []
    for a, b in ((h, y), far):
        h2, x, st = pkg.block_norm(a, b, want_stats=True, **par)
        g = pkg.block_norm_backward(a, b, st, dh_out=dh, dx=dx, **par)
        out.append([h2, x, st, g.dh, g.dy, g.dpre_weight, g.dpost_weight, g.dgate])
    assert all(torch.equal(a, b) for a, b in zip(*out))


def test_streams_and_graph_replays():
    T, D = 300, 1024
    par = dict(pre_weight=rand(D, seed=1), post_weight=rand(D, seed=2), gate=rand(D, seed=3),
               res_scale=rand(D, seed=4))
    h, y, dh, dx = (rand(T, D, seed=5 + i, dtype=B) for i in range(4))

    def step(stream=None):
        h2, x, st = pkg.block_norm(h, y, want_stats=True, stream=stream, **par)
        g = pkg.block_norm_backward(h, y, st, dh_out=dh, dx=dx, stream=stream, **par)
        return [h2, x, st, g.dh, g.dy, g.dpre_weight, g.dpost_weight, g.dgate, g.dres_scale]

    want = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = step(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph, other = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    with torch.cuda.graph(other):
        out2 = step()
    for seed in range(3):
        y.copy_(rand(T, D, seed=50 + seed, dtype=B))
        graph.replay()
        other.replay()
        torch.cuda.synchronize()
        want = step()
        assert all(torch.equal(a, b) for a, b in zip(out, want))
        assert all(torch.equal(a, b) for a, b in zip(out2, want))
