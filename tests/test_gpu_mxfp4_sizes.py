"""Rows longer than 2^32 values: the C ABI counts columns and matrix rows in 32
bits, and a size that does not fit is refused, not cut."""

import pytest
import torch

import sparse_moe_layer_latentmoe_amd as pkg

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
LONG = 2 ** 32 + 64


def refused(call):
    with pytest.raises(pkg.LmoeError) as e:
        call()
    assert e.value.status == pkg.LMOE_ERR_UNSUPPORTED


def test_rows_too_long_to_count():
    x = torch.zeros(1, LONG, dtype=torch.bfloat16, device=DEV)
    refused(lambda: pkg.quantize_mxfp4_rows(x))
    del x
    codes = torch.zeros(1, LONG // 2, dtype=torch.uint8, device=DEV)
    scales = torch.full((1, LONG // 32), 127, dtype=torch.uint8, device=DEV)
    refused(lambda: pkg.dequantize_mxfp4(codes, scales))


def test_products_with_too_many_rows():
    x = torch.zeros(1, 64, dtype=torch.uint8, device=DEV)
    xs = torch.full((1, 4), 127, dtype=torch.uint8, device=DEV)
    w, ws = x.expand(16, 64).contiguous(), xs.expand(16, 4).contiguous()
    rows = torch.zeros(2 ** 32 + 3, dtype=torch.int32, device=DEV)
    refused(lambda: pkg.mxfp4_matmul(x, xs, w, ws, rows=rows))
