#!/usr/bin/env python3
"""Times the cases of perf/operators.py and perf/more_operators.py through the package's operators.

  python perf/replay.py [CASE ...]      microseconds a call: from Python (calls one after another) and replayed
                                        from a CUDA graph, two input sets in turn
  python perf/replay.py --plain [CASE ...]  microseconds a call of the cases' plain forms, in elementary torch operations
  python perf/replay.py --twice CASE    the case called twice, 300 MB written between the calls, for a profiler
                                        (the second call's kernels begin on cold caches)
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from perf import more_operators, operators  # noqa: E402

CALLS = 20


def microseconds(fn, calls):
    """Device time of one of `calls` calls that fn() makes, warm."""
    fn()
    torch.cuda.synchronize()
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    start.record()
    fn()
    end.record()
    torch.cuda.synchronize()
    return start.elapsed_time(end) * 1e3 / calls


def time_case(operators, case):
    states = [operators.prepare(case, seed) for seed in (1, 2)]

    def run():
        for i in range(CALLS):
            operators.run(states[i % 2])

    called = microseconds(run, CALLS)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    return called, microseconds(lambda: (graph.replay(), graph.replay()), 2 * CALLS)


def time_plain(operators, case):
    states = [operators.prepare(case, seed) for seed in (1, 2)]
    calls = 4
    return microseconds(lambda: [operators.run(states[i % 2]) for i in range(calls)], calls)


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--twice", action="store_true")
    ap.add_argument("--plain", action="store_true")
    ap.add_argument("case", nargs="*")
    args = ap.parse_args()
    cases = {}
    for module in (operators, more_operators):
        module.own = not args.plain
        cases.update((c["name"], (module, c)) for c in module.listed())
    for name in args.case or cases:
        module, case = cases[name]
        if args.twice:
            state = module.prepare(case, 1)
            module.run(state)
            torch.empty(300 << 20, dtype=torch.uint8, device="cuda").zero_()
            module.run(state)
            torch.cuda.synchronize()
        elif args.plain:
            print("%-18s plain %8.2f us" % (name, time_plain(module, case)), flush=True)
        else:
            print("%-18s call %8.2f us   graph %8.2f us" % (name, *time_case(module, case)), flush=True)


if __name__ == "__main__":
    main()
