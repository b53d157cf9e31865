"""Times passes of the measured operators through the binding: the cases of
``perf/operators.py`` and further forms of the same operators (types, widths and
row counts that take other kernels).

    python3 profiles/time_operators.py [--only NAME,...] [--passes N]

prints, for each case, the time of a pass among others (events around rounds of
``N`` passes on one stream, the shortest of five rounds) and what it has to
move over that time.  Under a profiler ``--passes 10 --rounds 1`` gives ten
launches a kernel and round.
"""

import argparse
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)

import torch  # noqa: E402

import perf.operators as P  # noqa: E402
import sparse_moe_layer_latentmoe_amd as lmoe  # noqa: E402


def further():
    """Forms beside the listed cases."""
    out = []
    for d in (576, 1024, 2112, 4096, 6144, 8191, 8192, 16384):
        t = 4099 * 8192 // d
        out.append(P._norm(f"norm_f32_bf16_{d}", t, d, stream="f32", gate="full", train=True))
    out += [P._norm("norm_f32_f32_8192", 4099, 8192, stream="f32", dtype="f32", gate="full",
                    train=True),
            P._norm("norm_bf16_f32_8192", 4099, 8192, stream="bf16", dtype="f32", gate="full",
                    train=True),
            P._norm("norm_bf16_bf16_8192", 4099, 8192, gate="channel", train=True)]
    for t in (192, 1024, 2048):
        out.append(P._experts(f"experts_up_{t}", t, 22, 512, 5120, 2048, True))
        out.append(P._experts(f"experts_down_{t}", t, 22, 512, 2048, 5120, False))
    for m in (32, 64, 512, 2048):
        out.append(P._mm(f"matmul_{m}", m, 10240, 8192))
    out.append(P._mm("matmul_8192_f32", 8192, 10240, 8192, out="f32"))
    # weights as a checkpoint holds them -> codes and scales, once
    out.append({"name": "quantize_weight_512", "op": "weight", "shape": (512, 5120, 2048)})
    return out


def prepare(case):
    if case["op"] != "weight":
        return P.prepare(case, 1)
    n, *shape = case["shape"]
    w = torch.empty(n, *shape, dtype=torch.bfloat16, device="cuda")
    for i in range(n):
        w[i].normal_(0, 0.02)
    return w


def one(case, st):
    return lmoe.quantize_fp8_weight(st) if case["op"] == "weight" else P.run(st)


def moved(case):
    if case["op"] != "weight":
        return P.work(case)["bytes"]
    n = 1
    for d in case["shape"]:
        n *= d
    return 3 * n


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--only", default="")
    ap.add_argument("--passes", type=int, default=50)
    ap.add_argument("--rounds", type=int, default=5)
    a = ap.parse_args()
    P.own = True
    only = set(filter(None, a.only.split(",")))
    for case in P.listed() + further():
        if only and case["name"] not in only:
            continue
        st = prepare(case)
        one(case, st)
        torch.cuda.synchronize()
        best = float("inf")
        for _ in range(a.rounds):
            beg, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            beg.record()
            for _ in range(a.passes):
                one(case, st)
            end.record()
            torch.cuda.synchronize()
            best = min(best, beg.elapsed_time(end) * 1e3 / a.passes)
        print(f"{case['name']:24s} {best:10.2f} us  {moved(case) / best / 1e3:8.0f} GB/s", flush=True)
        del st
        torch.cuda.empty_cache()


if __name__ == "__main__":
    main()
