"""8-bit block-scaled matrices on the GPU against the float64 oracle.

Codes and scales are defined by correctly rounded fp32 steps, so they are
compared bit for bit.  A product: code products are exact in fp32; a block's
128 of them are added (at worst one rounding of 2^-23 each, were the matrix
core to truncate; the 8-bit instruction, which bf16 results take, was measured
at 2^-15.9 of the magnitudes), its sum is scaled (3 * 2^-24) and added to
K / 128 others: at most (128 * 2 + 3 + K / 128) * 2^-24 < 2^-15 of the sum of
the terms' magnitudes for K up to 65536; then one rounding to the output
type.  fp32 results have a narrower bound of their own below."""

import numpy as np
import pytest
import torch

import sparse_moe_layer_latentmoe_amd as pkg
from oracle import operators as R

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F, B = torch.float32, torch.bfloat16


def rand(*shape, seed, dtype=F, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * std).to(dtype).to(DEV)


def bits(q):
    return q.view(torch.uint8).cpu().numpy()


def check_quantize(x):
    q, s = pkg.quantize_fp8(x)
    wq, ws = R.quantize_fp8(x.float().cpu().numpy())
    assert np.array_equal(s.cpu().numpy(), ws)
    assert np.array_equal(bits(q), wq)


@pytest.mark.parametrize("dtype", [B, F])
@pytest.mark.parametrize("T,K", [(1, 1), (1, 128), (3, 100), (7, 136), (17, 640), (33, 1000),
                                 (5, 129), (64, 2048), (2, 10240)])
def test_activations(T, K, dtype):
    x = rand(T, K, seed=T + K, dtype=dtype) * torch.exp(3 * rand(T, 1, seed=1)).to(dtype)
    check_quantize(x)


def test_activation_values_at_the_edges():
    x = rand(12, 256, seed=3)
    x[0] = 0
    x[1] *= 1e-42                       # denormal: the scale stops at 2^-126
    x[2] *= 1e-30                       # small scale: the division itself
    x[3] *= 1e36
    x[4, :] = torch.finfo(F).max
    x[5, :128] = torch.linspace(-448, 448, 128, device=DEV)     # scale 1: ties among them
    x[6, :128] = torch.arange(128, device=DEV) * 0.0009765625   # subnormal codes and their ties
    x[6, 127] = 448.0
    x[7, 1:] = 0
    x[8] = -0.0
    x[9] = 2.0 ** -126 * 448
    check_quantize(x)
    # the largest fp32 number is infinite in bf16: its largest finite one there
    big = torch.finfo(B).max
    check_quantize(x.clamp(-big, big).to(B))


def test_strided_and_unaligned_activations():
    wide = rand(19, 700, seed=4, dtype=B)
    for sl in (np.s_[:, 8:136], np.s_[:, 3:259], np.s_[:, 1:2], np.s_[:, 0:640], np.s_[2:, 16:529]):
        check_quantize(wide[sl])
    check_quantize(wide.float()[:, 4:260])


def test_rows_further_apart_than_32_bits():
    x = torch.empty(2, 2 ** 31, dtype=B, device=DEV)[:, :300]
    x.copy_(rand(2, 300, seed=3))
    check_quantize(x)


@pytest.mark.parametrize("dtype", [B, F])
@pytest.mark.parametrize("shape", [(128, 128), (16, 128), (1, 1), (144, 256), (300, 200), (3, 48, 384),
                                   (2, 2, 130, 129)])
def test_weights(shape, dtype):
    w = rand(*shape, seed=sum(shape), dtype=dtype, std=0.02)
    q, s = pkg.quantize_fp8_weight(w)
    assert q.shape == w.shape
    flat = w.float().cpu().numpy().reshape(-1, *shape[-2:])
    fq, fs = bits(q).reshape(flat.shape), s.cpu().numpy().reshape(flat.shape[0], *s.shape[-2:])
    for i in range(flat.shape[0]):
        wq, ws = R.quantize_fp8(flat[i], 128)
        assert np.array_equal(fs[i], ws) and np.array_equal(fq[i], wq)


def operands(X, N, K, G=None, seed=0):
    xc, xs = pkg.quantize_fp8(rand(X, K, seed=seed))
    wc, ws = pkg.quantize_fp8_weight(rand(*((N, K) if G is None else (G, N, K)), seed=seed + 1,
                                          std=0.02))
    return xc, xs, wc, ws


def check(ops, offsets=None, rows=None, dtype=B):
    xc, xs, wc, ws = ops
    M = xc.shape[0] if rows is None else len(rows)
    N = wc.shape[-2]
    i32 = lambda v: None if v is None else torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    out = torch.full((M, N), 7.0, dtype=dtype, device=DEV)
    y = pkg.fp8_matmul(xc, xs, wc, ws, offsets=i32(offsets), rows=i32(rows), out=out)
    want, mag, done = R.fp8_matmul(bits(xc), xs.cpu().numpy(), bits(wc), ws.cpu().numpy(),
                                   offsets, None if rows is None else np.asarray(rows))
    got = y.double().cpu().numpy()
    assert np.all(got[~done] == 7.0)
    unit = torch.finfo(dtype).eps / 2
    err = np.abs(got - want)[done]
    ok = (2.0 ** -15 * (1 + unit) * mag + unit * np.abs(want))[done]
    assert np.all(err <= ok), float((err / np.maximum(ok, 1e-300)).max())
    return y


@pytest.mark.parametrize("dtype", [B, F])
@pytest.mark.parametrize("M", [1, 2, 15, 16, 17, 33, 64])
@pytest.mark.parametrize("N,K", [(16, 128), (48, 256), (144, 1152), (400, 640)])
def test_few_rows(M, N, K, dtype):
    check(operands(M, N, K, seed=M + N + K), dtype=dtype)


@pytest.mark.parametrize("dtype", [B, F])
@pytest.mark.parametrize("M,N,K", [(65, 16, 128), (100, 272, 256), (187, 512, 384), (256, 256, 512),
                                   (257, 128, 640), (300, 400, 1152), (511, 784, 896),
                                   (130, 1040, 2048)])
def test_many_rows(M, N, K, dtype):
    check(operands(M, N, K, seed=M + N + K), dtype=dtype)


@pytest.mark.parametrize("groups", [0, 7])
@pytest.mark.parametrize("M,K", [(9, 128), (40, 128), (300, 128), (300, 1024), (900, 512),
                                 (2100, 256), (4500, 128)])
def test_fp32_results_are_fp32_sums(M, K, groups):
    """fp32 results come from fp32 sums, through every kind of tile: each of a
    block's 128 additions, the two scalings and the addition to the running sum
    rounds by at most 2^-24 of a partial sum, which is at most the sum of the
    magnitudes."""
    xc, xs, wc, ws = operands(M, 256, K, groups or None, seed=M)
    off = None
    if groups:
        off = torch.tensor([M * i // groups for i in range(groups + 1)], dtype=torch.int32,
                           device=DEV)
    y = pkg.fp8_matmul(xc, xs, wc, ws, offsets=off, out_dtype=F)
    want, mag, _ = R.fp8_matmul(bits(xc), xs.cpu().numpy(), bits(wc), ws.cpu().numpy(),
                                None if off is None else off.tolist(), None)
    err = np.abs(y.double().cpu().numpy() - want)
    assert np.all(err <= (128 + 3 * (K // 128)) * 2.0 ** -24 * mag), float((err / mag).max())


def test_long_k():
    check(operands(70, 32, 65536, seed=1))
    check(operands(5, 32, 65536, seed=2))


def offsets_of(counts):
    return [0] + list(np.cumsum(counts))


@pytest.mark.parametrize("dtype", [B, F])
@pytest.mark.parametrize("counts", [[1], [0, 3, 0, 1], [16, 17, 1, 0, 40], [0, 0, 0, 5],
                                    [200, 0, 129, 64, 1, 300], [128, 256, 127, 257], [600]])
@pytest.mark.parametrize("N,K", [(16, 128), (272, 384), (528, 256)])
def test_groups(counts, N, K, dtype):
    M, G = sum(counts), len(counts)
    check(operands(M, N, K, G, seed=M + N), offsets_of(counts), dtype=dtype)
    g = np.random.default_rng(M)
    check(operands(37, N, K, G, seed=M + N), offsets_of(counts), list(g.integers(0, 37, M)),
          dtype=dtype)


def test_many_groups():
    g = np.random.default_rng(3)
    for mean in (0.5, 3, 40):
        counts = g.poisson(mean, 1024)
        check(operands(int(counts.sum()), 32, 128, 1024, seed=9), offsets_of(counts))


def test_rows_of_no_group_and_bad_indices():
    ops = operands(90, 48, 256, 3, seed=11)
    check(ops, [4, 10, 10, 70])                       # rows before and behind the groups
    check(ops, [0, 0, 0, 0])
    check(operands(30, 48, 256, 3, seed=12), [0, 40, 41, 100],
          [-1, 30, 2 ** 31 - 1, -2 ** 31] + [i % 30 for i in range(96)])
    check(operands(30, 48, 256, seed=12)[:2] + operands(30, 48, 256, seed=12)[2:],
          rows=[29, -7, 3, 3, 30] + [5] * 200)
    # offsets past the rows are cut; those that do not ascend stay in bounds
    xc, xs, wc, ws = ops
    check(ops, [0, 50, 95, 200])
    for bad in ([50, 20, 90, 10], [-5, 90, -1, 90], [2 ** 31 - 1, -2 ** 31, 0, 90], [0, 90, 0, 90]):
        guard = torch.full((92, 48), 7.0, dtype=B, device=DEV)
        pkg.fp8_matmul(xc, xs, wc, ws, torch.tensor(bad, dtype=torch.int32, device=DEV),
                       out=guard[1:91])
        torch.cuda.synchronize()
        assert bool((guard[0] == 7).all()) and bool((guard[91] == 7).all())


def test_many_offsets_at_the_ends_of_their_type():
    """Each pair asks for 2^31 rows if taken at its word."""
    ops = operands(90, 48, 256, 400, seed=11)
    guard = torch.full((92, 48), 7.0, dtype=B, device=DEV)
    bad = [2 ** 31 - 1, -2 ** 31] * 200 + [90]
    for off in (bad, [1] + bad[:-1]):
        pkg.fp8_matmul(*ops, torch.tensor(off, dtype=torch.int32, device=DEV), out=guard[1:91])
        torch.cuda.synchronize()
        assert bool((guard[0] == 7).all()) and bool((guard[91] == 7).all())


def test_no_rows():
    xc, xs, wc, ws = operands(1, 32, 128)
    assert pkg.fp8_matmul(xc[:0], xs[:0], wc, ws).shape == (0, 32)
    none = torch.zeros(0, dtype=torch.int32, device=DEV)
    assert pkg.fp8_matmul(xc, xs, wc, ws, rows=none).shape == (0, 32)
    q, s = pkg.quantize_fp8(rand(0, 256, seed=0))
    assert q.shape == (0, 256) and s.shape == (0, 2)


def test_same_bits_on_another_stream_and_in_two_graphs():
    counts = [70, 0, 300, 5]
    off = torch.tensor(offsets_of(counts), dtype=torch.int32, device=DEV)
    x = rand(sum(counts), 512, seed=1, dtype=B)
    w, ws = pkg.quantize_fp8_weight(rand(4, 320, 512, seed=2, std=0.02))

    def step(stream=None):
        q, s = pkg.quantize_fp8(x, stream=stream)
        return pkg.fp8_matmul(q, s, w, ws, off, stream=stream)

    want = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = step(side)
    side.synchronize()
    assert torch.equal(got, want)
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1):
        y1 = step()
    with torch.cuda.graph(g2):
        y2 = step()
    for seed in range(3):
        x.copy_(rand(*x.shape, seed=20 + seed, dtype=B))
        g1.replay()
        g2.replay()
        torch.cuda.synchronize()
        want = step()
        assert torch.equal(y1, want) and torch.equal(y2, want)
