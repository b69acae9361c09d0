"""Child process of tests/test_gpu_table_run.py (not a test module): a fresh
process whose first table calls, after zs_init, are captured."""
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)
sys.path.insert(0, os.path.join(ROOT, "tests"))

import torch  # noqa: E402

import fsdp_sharded_optimizer_zero_amd as Z  # noqa: E402
from test_gpu_table_run import SHAPES, Calls  # noqa: E402


def main():
    torch.cuda.set_device(0)
    calls = [Calls(*shape, seed=30 + i) for i, shape in enumerate(SHAPES)]
    again = [Calls(*shape, seed=30 + i) for i, shape in enumerate(SHAPES)]
    Z.zs_init()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for c in calls:
            c.run()
    for k in range(3):
        graph.replay()
        got = [c.snapshot() for c in calls]
        for c, g in zip(again, got):
            c.run()
            want = c.snapshot()
            assert all(torch.equal(g[n], want[n]) for n in g), f"replay {k}"
    print("capture-first ok", flush=True)


main()
