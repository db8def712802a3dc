"""Device time of the decoding step's operators among other calls: calls captured into a graph, over one set of
operands ("warm": what fits stays in L2) and over as many as pass L2 three times ("cold": every call reads HBM, as the
layers of a model do).

    python perf/graph_times.py [name ...]

The cases are those of perf/more_operators.py and some forms beside them.
"""
import os
import statistics
import sys

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))

import torch  # noqa: E402

from perf import more_operators as ops  # noqa: E402

L2 = 129 << 20
CALLS, REPLAYS = 24, 7


def cases():
    yield from ops.listed()
    attend, product = ops._attend, ops._product
    # fp32 output at length, both head sizes
    yield dict(attend(32, 1, 4096, 32, 8, 128, 64, "chain", "f32"), name="attend_step_f32")
    yield dict(attend(32, 1, 4096, 32, 8, 64, 64, "chain", "f32"), name="attend_step_f32_64")
    yield dict(attend(16, 64, 8192, 32, 8, 128, 64, "tree", "f32"), name="attend_tree_f32")
    yield dict(attend(1, 1, 262143, 32, 8, 128, 128, "chain", "f32", False), name="attend_long_f32")
    yield dict(attend(4, 500, 2000, 28, 4, 128, 32, "chain", "f32"), name="attend_chunk_f32")
    # more rows at ordinary sizes
    yield dict(product(32, 8192, 8192, 128, "none", "bf16"), name="product_32")
    yield dict(product(64, 8192, 8192, 128, "none", "bf16"), name="product_64")
    yield dict(product(64, 4096, 4096, 64, "none", "bf16"), name="product_64_mid")


def per_call(states):
    """Microseconds a call, the states one after the other."""
    calls = max(CALLS, len(states))
    for s in states[:2]:
        ops.run(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for i in range(calls):
            ops.run(states[i % len(states)])
    times = []
    for i in range(3 + REPLAYS):
        start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        start.record()
        graph.replay()
        end.record()
        torch.cuda.synchronize()
        if i >= 3:
            times.append(start.elapsed_time(end) * 1000.0 / calls)
    return statistics.median(times)


def main(names):
    ops.own = True
    for case in cases():
        if names and case["name"] not in names:
            continue
        size = ops.work(case)["bytes"]
        many = min(64, max(2, -(-3 * L2 // size)))
        states = [ops.prepare(case, seed) for seed in range(1, many + 1)]
        print("%-20s warm %8.2f us   cold %8.2f us (%d sets%s)" % (
            case["name"], per_call(states[:1]), per_call(states), many, "" if many * size >= 3 * L2 else ", which L2 holds in part"), flush=True)
        del states


if __name__ == "__main__":
    main(sys.argv[1:])
