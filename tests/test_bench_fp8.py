"""The benchmark's workloads of the layer with FP8 experts: names and byte
counts by hand."""

import pytest

import bench
import lmoe_inputs as li


@pytest.mark.parametrize("name,layer,fmt,block", [
    ("decode", "decode", "", False), ("decode_fp8", "decode", "fp8", False),
    ("mtp_verify_fp8", "mtp_verify", "fp8", False), ("prefill_fp8", "prefill", "fp8", False),
    ("prefill_mxfp4", "prefill", "mxfp4", False), ("decode_mxfp4_block", "decode", "mxfp4", True)])
def test_names(name, layer, fmt, block):
    assert name in bench.WORKLOADS
    wl, f, b = bench.parse_workload(name)
    assert (wl.name, f, b) == (layer, fmt, block)
    assert ("FP8" in bench.describe(name, wl.shape, wl.tokens, f, b)) == (fmt == "fp8")


def test_decode_batch_expert_bytes_by_hand():
    b, _ = bench.stage_work(li.FULL, 32, 375, bench.FP8_WEIGHT_BYTES,
                            expert_row_bytes=bench.FP8_ROW_BYTES)
    # a byte per weight, 4 per 128 x 128 block; codes in and out with 4 per 128
    weights = 375 * 5120 * 2048 + 375 * (5120 // 128) * (2048 // 128) * 4
    assert b["expert_up"] == weights + 704 * (2048 + 5120) + 704 * (16 + 40) * 4
    assert b["expert_down"] == weights + 704 * 5120 + 704 * 40 * 4 + 704 * 2048 * 2
