"""Times of the products' cases (perf/operators.py) on this GPU.

    python perf/times.py [--only NAME,NAME] [--draw N] [--seed S]

For each case, over three sets of inputs in turn: `device`, microseconds a call in
a CUDA graph of twelve; `call`, microseconds a call from Python, one after another;
both by CUDA events, the least of five runs after a warm-up.  `floor` is the larger
of the case's bytes and its operations at this GPU's measured rates (with the MXFP8
instruction at twice the bf16 rate).  Where power bounds a call the clock drops, so
that the figures of large calls move by some percent between machines.
"""
import argparse
import json
import os
import random
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path[:0] = [ROOT, os.path.join(ROOT, "perf")]
import torch  # noqa: E402

import operators  # noqa: E402

SETS, CALLS, RUNS = 3, 12, 5


def rates():
    """Bytes and bf16 operations a second."""
    try:
        with open(os.path.join(ROOT, "MEASURED_PEAKS.json")) as f:
            d = json.load(f)
        return d["hbm_gbs"] * 1e9, d["bf16_tflops"] * 1e12
    except (OSError, KeyError, ValueError):
        return 6.8e12, 1.9e15


def least_us(run, calls):
    """Microseconds of one of the `calls` calls that run() makes."""
    run()
    times = []
    for _ in range(RUNS):
        torch.cuda.synchronize()
        start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        start.record()
        run()
        end.record()
        end.synchronize()
        times.append(start.elapsed_time(end) * 1e3 / calls)
    return min(times)


def measure(case, seed):
    states = [operators.prepare(case, seed + i) for i in range(SETS)]

    def calls(n):
        for i in range(n):
            operators.run(states[i % SETS])

    calls(SETS)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls(CALLS)
    replays = max(1, int(20e3 / (CALLS * least_us(graph.replay, CALLS))))

    def replay():
        for _ in range(replays):
            graph.replay()

    device = least_us(replay, CALLS * replays)
    return device, least_us(lambda: calls(CALLS * replays), CALLS * replays)


def main():
    p = argparse.ArgumentParser()
    p.add_argument("--only", default="")
    p.add_argument("--draw", type=int, default=0)
    p.add_argument("--seed", type=int, default=0)
    args = p.parse_args()
    operators.own = True
    rng = random.Random(args.seed)
    cases = operators.listed() + [{**operators.draw(rng), "name": f"draw_{i}"} for i in range(args.draw)]
    only = set(filter(None, args.only.split(",")))
    bytes_s, flops_s = rates()
    print(f"{'case':<20}{'floor us':>10}{'device us':>11}{'call us':>9}{'GB/s':>8}{'TFLOP/s':>9}  (device)")
    for case in cases:
        if only and case["name"] not in only:
            continue
        work = operators.work(case)
        floor = max(work["bytes"] / bytes_s, work["flops"] / (2 * flops_s)) * 1e6
        device, call = measure(case, args.seed)
        print(f"{case['name']:<20}{floor:>10.2f}{device:>11.2f}{call:>9.2f}{work['bytes'] / device / 1e3:>8.0f}"
              f"{work['flops'] / device / 1e6:>9.0f}", flush=True)


if __name__ == "__main__":
    main()
