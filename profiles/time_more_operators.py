"""Times passes of the 4-bit operators and of the sparse layer for a few tokens
through the binding: the cases of ``perf/more_operators.py`` and further forms
(row and token counts that take other kernels).

    python3 profiles/time_more_operators.py [--only NAME,...] [--passes N] [--rounds N]

prints, for each case, the time of a pass among others (events around rounds of
``N`` passes on one stream, the shortest of the rounds) and what it has to move
over that time.  Under a profiler ``--passes 10 --rounds 1`` gives ten launches a
kernel and round.
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
        for t in (2, 4, 8, 16):
            out.append(P._tokens(f"tokens_{t}_{fmt}", t, 512, 22, 2048, 5120, fmt=fmt, dtype="f32"))
    return out


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
        st = P.prepare(case, 1)
        P.run(st)
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
        w = P.work(case)
        print(f"{case['name']:24s} {best:10.2f} us  {w['bytes'] / best / 1e3:8.0f} GB/s"
              f"  {w['flops'] / best / 1e6:8.1f} TFLOP/s", flush=True)
        del st
        torch.cuda.empty_cache()


if __name__ == "__main__":
    main()
