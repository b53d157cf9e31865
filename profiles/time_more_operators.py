"""Times passes of the 4-bit operators and of the sparse layer for a few tokens
through the binding: the cases of ``perf/more_operators.py`` and further forms
(row and token counts that take other kernels).

    python3 profiles/time_more_operators.py [--only NAME,...] [--passes N] [--rounds N]

prints, for each case, the time of a pass among others (events around rounds of
``N`` passes on one stream, the shortest of the rounds) and what it has to move
over that time (a sparse layer: with the experts that its tokens used).  Under a
profiler ``--passes 10 --rounds 1`` gives ten launches a kernel and round.
"""

import argparse
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)

import torch  # noqa: E402

import perf.more_operators as P  # noqa: E402


def further():
    """Forms beside the listed cases."""
    out = [P._mm(f"matmul_{m}", m, 10240, 8192) for m in (8, 16, 32, 64, 512, 2048)]
    out.append(P._mm("matmul_8192_f32", 8192, 10240, 8192, out="f32"))
    for t in (192, 1024, 2048):
        out.append(P._grouped(f"experts_up_{t}", t, 22, 512, 5120, 2048, True))
        out.append(P._grouped(f"experts_down_{t}", t, 22, 512, 2048, 5120, False))
    for fmt in ("bf16", "fp8", "mxfp4"):
        for t in (1, 2, 4, 8, 16):
            out.append(P._tokens(f"tokens_{t}_{fmt}", t, 512, 22, 2048, 5120, fmt=fmt, dtype="f32"))
        # gated experts of the same width
        out.append(P._tokens(f"gated_1_{fmt}", 1, 512, 22, 2048, 5120, fmt=fmt, act="swiglu"))
        # a wide shared expert, and experts that all tokens take
        for t, x in ((8, "bf16"), (8, "f32"), (16, "bf16"), (16, "f32")):
            out.append(P._tokens(f"shared_{t}_{fmt}_{x}", t, 8, 2, 8192, 1024, fmt=fmt,
                                 shared=10240, dtype=x))
        for t in (8, 16):
            out.append(P._tokens(f"crowded_{t}_{fmt}", t, 8, 8, 2048, 2048, fmt=fmt, act="swiglu",
                                 score="softmax", scale=1.0))
    # one expert takes every row
    out.append(dict(P._grouped("experts_one_of_64", 80, 8, 64, 5120, 2048, True), crowd=True))
    return out


def prepare(case):
    st = P.prepare(case, 1)
    if case.get("crowd"):
        st["offsets"][1:] = st["offsets"][-1]
    return st


def moved(case, out):
    """Bytes of a pass: a sparse layer's with the experts its tokens used."""
    if case["op"] != "tokens":
        return P.work(case)["bytes"]
    alone = P.work(dict(case, tokens=1, top_k=1))["bytes"]
    two = P.work(dict(case, tokens=1, top_k=2))["bytes"]
    rest = P.work(dict(case, top_k=0))["bytes"]
    used = len(set(out["experts"].flatten().tolist()))
    return rest + used * (two - alone)


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
        bytes_ = moved(case, P.run(st))
        torch.cuda.synchronize()
        best = float("inf")
        for _ in range(a.rounds):
            beg, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            beg.record()
            for _ in range(a.passes):
                P.run(st)
            end.record()
            torch.cuda.synchronize()
            best = min(best, beg.elapsed_time(end) * 1e3 / a.passes)
        print(f"{case['name']:24s} {best:10.2f} us  {bytes_ / best / 1e3:8.0f} GB/s"
              f"  {P.work(case)['flops'] / best / 1e6:8.1f} TFLOP/s", flush=True)
        del st
        torch.cuda.empty_cache()


if __name__ == "__main__":
    main()
