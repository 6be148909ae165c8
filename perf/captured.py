"""Times of the operators' calls: `python perf/captured.py [NAME ...]`.

For each listed case of operators.py (or those named) the microseconds of one call
in a captured CUDA graph -- the GPU's time, with the launch over the tail of the
call before -- and of one call among eager calls through the binding, which the
host bounds where it is slower.  Calls go over as many states of different seeds as
outgrow L2 (at most 16), so that a call finds none of its inputs there unless the
case is too small for that.
"""
from __future__ import annotations

import sys
from pathlib import Path

sys.path.insert(0, str(Path(__file__).resolve().parent.parent))

import torch  # noqa: E402

from perf import operators  # noqa: E402

L2_BYTES = 129 << 20


def _us(run, calls: int) -> float:
    """Microseconds a call of the fastest of five repeats of run(), which makes `calls` of them."""
    best = float("inf")
    for _ in range(5):
        start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        torch.cuda.synchronize()
        start.record()
        run()
        end.record()
        end.synchronize()
        best = min(best, start.elapsed_time(end) * 1e3 / calls)
    return best


def measure(case) -> tuple[float, float]:
    """(captured, eager) microseconds a call."""
    count = max(2, min(16, 1 + 2 * L2_BYTES // max(1, operators.work(case)["bytes"])))
    states = [operators.prepare(case, seed) for seed in range(count)]

    def each():
        for s in states:
            operators.run(s)

    for _ in range(3):
        each()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        each()
    graph.replay()
    rounds = max(1, 200 // count)

    def repeat(f):
        for _ in range(rounds):
            f()

    return _us(lambda: repeat(graph.replay), rounds * count), _us(lambda: repeat(each), rounds * count)


def main(names) -> None:
    operators.own = True
    for case in operators.listed():
        if not names or case["name"] in names:
            floor = operators.work(case)["bytes"]
            print("{:20s} captured {:8.2f} us  eager {:8.2f} us  {:10.3f} MB".format(
                case["name"], *measure(case), floor / 1e6), flush=True)


if __name__ == "__main__":
    main(sys.argv[1:])
