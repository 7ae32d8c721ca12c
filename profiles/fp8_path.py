"""The passes that the 8-bit path's profiles are taken of: the workloads of
perf/operators.py through the library, and a few calls beside them.

    cd /tmp && export TMPDIR=/tmp        ($REPO is the repository root)
    rocprofv3 --kernel-trace --stats -d OUT -o kt -- python3 $REPO/profiles/fp8_path.py
    python3 $REPO/profiles/fp8_path.py --summarise OUT/kt_results.db

Every pass takes the next of several states, enough that together they move
512 MiB (at most 128: the smallest calls' inputs stay in the last-level cache,
256 MB, all the same).  Prints each case as it begins, with its states.
--summarise prints each case's kernels from a trace: threads, registers, LDS
and times, after a first round over the case's states.
"""

import argparse
import os
import re
import sqlite3
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)

import torch  # noqa: E402

import vq_compressed_linear_amd as hx  # noqa: E402
from perf import operators as ops  # noqa: E402

ops.own = True
APART = 2  # launches of torch's own that may stand between two of a case's (scales that are laid out for a call)


def turns(name, make, run, moved, passes):
    """`passes` runs, each on the next of enough states."""
    n = min(128, max(2, -(-(512 << 20) // max(1, int(moved)))))
    print("%s: %d states of %.1f MB, %d passes" % (name, n, moved / 1e6, passes), flush=True)
    states, mark = [make(i) for i in range(n)], torch.empty(1, device="cuda")
    for count in (n, passes):  # a round over all states, then the passes that --summarise takes
        for _ in range(APART + 1):
            mark.zero_()
        for i in range(count):
            run(states[i % n])
        torch.cuda.synchronize()


def square(y):
    """8192^3 from rows of e4m3."""
    n = 8192
    s = torch.full((n, 64), 127, dtype=torch.uint8, device="cuda").view(ops.E8M0)

    def make(seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        x, w = [torch.randn(n, n, generator=g, device="cuda").to(ops.E4M3) for _ in range(2)]
        return x, w, s[: n // 128].contiguous(), torch.empty(n, n, dtype=y, device="cuda")

    return make, lambda t: hx.hxq_linear_fwd_fp8(t[0], s, t[1], t[2], None, t[3]), 2 * n * n + n * n * y.itemsize


def one_row(n, k):
    """One bf16 row through a layer of n x k."""
    def make(seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        w = torch.randn(n, k, generator=g, device="cuda").to(ops.E4M3)
        s = torch.full((-(-n // 128), hx.fp8_scale_columns(k)), 127, dtype=torch.uint8, device="cuda").view(ops.E8M0)
        return torch.randn(1, k, generator=g, device="cuda").bfloat16(), w, s, torch.empty(1, n, device="cuda")

    return make, lambda t: hx.hxq_linear_fwd_fp8(t[0], None, t[1], t[2], None, t[3]), n * k


def weight(transposed):
    """gate|up's weight from bf16 to e4m3."""
    n, k = 22016, 2048

    def make(seed):
        def new(rows, cols):
            return (torch.empty(rows, cols, dtype=ops.E4M3, device="cuda"),
                    torch.empty(rows // 128, hx.fp8_scale_columns(cols), dtype=ops.E8M0, device="cuda"))

        g = torch.Generator(device="cuda").manual_seed(seed)
        w = torch.randn(n, k, generator=g, device="cuda").bfloat16()
        return (w, *new(n, k), *(new(k, n) if transposed else (None, None)))

    return make, lambda t: hx.hxq_quant_fp8_weight(*t), n * k * (4 if transposed else 3)


EXTRA = {
    "square-bf16": lambda: square(torch.bfloat16),
    "square-f32": lambda: square(torch.float32),
    "row-2048x2048": lambda: one_row(2048, 2048),
    "row-8512x2048": lambda: one_row(8512, 2048),
    "row-2048x11008": lambda: one_row(2048, 11008),
    "weight": lambda: weight(False),
    "weight-transposed": lambda: weight(True),
}


def summarise(path):
    """Each second run of the library's kernels (torch's lie between a case's first round and its passes, and
    between two cases), by kernel."""
    rows = sqlite3.connect(path).execute("select name, grid_x, vgpr_count, lds_size, duration from kernels order by start")
    cases, apart = [], APART + 1
    for name, *rest in rows:
        if "hxq::" not in name:
            apart += 1
            continue
        if apart > APART:
            cases.append({})
        apart = 0
        name = re.sub(r"\(hxq::\w+.*|\(void const\*.*|\(float const\*.*", "", name)
        name = re.sub(r"^void |hxq::|\(anonymous namespace\)::", "", name)
        cases[-1].setdefault((name, *rest[:3]), []).append(rest[3] / 1e3)
    out = ["%-66s %9s %5s %7s %4s %10s %10s" % ("kernel", "threads", "vgpr", "lds", "n", "median us", "min us")]
    for case in cases[1::2]:
        out.append("")
        for (name, threads, vgpr, lds), t in case.items():
            t = sorted(t)
            out.append("%-66s %9d %5d %7d %4d %10.2f %10.2f" % (name[:66], threads, vgpr, lds, len(t), t[len(t) // 2], t[0]))
    return "\n".join(out)


def main():
    cases = {c["name"]: c for c in ops.listed()}
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--only", default="", help="comma-separated, of: %s" % ", ".join([*cases, *EXTRA]))
    ap.add_argument("--passes", type=int, default=24)
    ap.add_argument("--summarise", metavar="DB")
    args = ap.parse_args()
    if args.summarise:
        print(summarise(args.summarise))
        return
    for name in args.only.split(",") if args.only else [*cases, *EXTRA]:
        if name in EXTRA:
            turns(name, *EXTRA[name](), args.passes)
        else:
            case = cases[name]
            turns(name, lambda i: ops.prepare(case, i), ops.run, ops.work(case)["bytes"], args.passes)
        torch.cuda.empty_cache()


if __name__ == "__main__":
    main()
