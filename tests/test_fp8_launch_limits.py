"""8-bit products too large for one launch (2^32 threads) are refused as
unsupported, before any HIP call, by the operator and by the layer; those next
to the limit are not."""

import pytest

import lmoe_inputs as li
import sparse_moe_layer_latentmoe_amd as pkg

FAKE = 0x10000000     # never dereferenced


@pytest.fixture(scope="module")
def lib():
    return pkg.load_library()


def args(**kw):
    a = pkg.LmoeFp8MatmulArgs()
    at = lambda i: FAKE + (i << 44)  # noqa: E731
    for k, v in dict(x=at(1), x_scales=at(2), w=at(3), w_scales=at(4), rows=at(5), offsets=at(6),
                     y=at(7), y_type=1, n_groups=1, M=1 << 24, x_rows=1, N=4096, K=32896).items():
        setattr(a, k, v)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


# streamed tiles of 16 rows: (1 + M / 16 + 1) * N / 64 work-groups of 256 threads
@pytest.mark.parametrize("kw,fits", [
    (dict(), False), (dict(N=1024), False), (dict(N=960), True), (dict(M=1 << 20), True),
    (dict(M=1 << 22, N=4096), False), (dict(M=1 << 22, N=3968), True), (dict(y_type=0), False),
    (dict(K=32768), True), (dict(N=1 << 20, M=1 << 17), False),
    (dict(n_groups=0, offsets=None, rows=None, x_rows=1 << 24, N=1 << 20, K=128), False),
    (dict(n_groups=0, offsets=None, rows=None, x_rows=1 << 24, N=1 << 14, K=128), True)])
def test_products(lib, kw, fits):
    a = args(**kw)
    if fits:
        # no GPU is asked: the workspace is what is missing
        if kw.get("n_groups", 1):
            assert lib.lmoe_fp8_matmul_workspace_size(a) > 0
            assert lib.lmoe_fp8_matmul(a, None, 0, None) == pkg.LMOE_ERR_WORKSPACE
    else:
        assert lib.lmoe_fp8_matmul_workspace_size(a) == 0
        assert lib.lmoe_fp8_matmul(a, FAKE + (9 << 44), 1 << 40, None) == pkg.LMOE_ERR_UNSUPPORTED


def test_streamed_layer():
    shape = li.LayerShape(256, 128, 64, 32, 2048, 512, 5.0)
    # 2^22 tokens x 32 / 16 tiles, 16 work-groups of 256 threads each
    for tokens, fits in (((1 << 22), False), ((1 << 18), True)):
        cfg = pkg.make_config(shape, tokens, pkg.PATH_STREAM, pkg.EXPERTS_FP8)
        assert (pkg.workspace_size(cfg) > 0) == fits
    assert pkg.workspace_size(pkg.make_config(shape, 1 << 22, pkg.PATH_AUTO, pkg.EXPERTS_FP8)) > 0
    assert pkg.workspace_size(pkg.make_config(shape, 1 << 22, pkg.PATH_STREAM)) > 0
