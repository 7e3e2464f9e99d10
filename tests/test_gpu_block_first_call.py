"""The first call of a process may be one that is captured: what the kernels with clusters of
16 CTAs ask the device once, they ask then."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = """
import torch
import stream_compaction_gb300 as sc
ids = torch.randint(-1, 64, (20000, 2), device="cuda")
x, g, dy = (torch.randn(1, 6000, 64, device="cuda", dtype=torch.bfloat16) for _ in range(3))
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    order = sc.expert_sort(ids, 64)
    saved = sc.gated_scan_saved(x)
    y = sc.gated_scan(x, g, saved=saved)
    grads = sc.gated_scan_grad(dy, x, g, saved=saved)
graph.replay()
torch.cuda.synchronize()
saved2 = sc.gated_scan_saved(x)
want = [*sc.expert_sort(ids, 64), sc.gated_scan(x, g, saved=saved2), *sc.gated_scan_grad(dy, x, g, saved=saved2).values()]
assert all(torch.equal(a, b) for a, b in zip([*order, y, *grads.values()], want))
print("the same")
"""


def test_captured():
    made = subprocess.run([sys.executable, "-c", PROGRAM], capture_output=True, text=True, cwd=ROOT, timeout=300)
    assert made.returncode == 0 and "the same" in made.stdout, made.stderr[-2000:]
