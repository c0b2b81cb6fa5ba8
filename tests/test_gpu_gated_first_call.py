"""A process whose first calls of the gated recurrence and the group norm are captured into a graph: what launches ask of the
device for the first time is asked during the capture."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

PROGRAM = """
import torch
import kimi_delta_attention_chunk_gb300 as kda

C, T = 512, 3000
rows = [torch.randn(1, T, C, device="cuda").to(torch.bfloat16) for _ in range(5)]
x, r, i, z, dy = rows
lam = torch.linspace(-6.0, -2.0, C, device="cuda")
cu = torch.tensor([0, 1200, 1201, T], dtype=torch.int32, device="cuda")
w = torch.randn(C, device="cuda")

def work():
    got = []
    for offsets in (None, cu):
        got += kda.gated_scan_fwd(x, r, i, lam, z=z, cu_seqlens=offsets)
        got += [v for v in kda.gated_scan_bwd(x, r, i, lam, dy, z=z, cu_seqlens=offsets).values() if v is not None]
        got.append(kda.group_norm_fwd(x, 8, weight=w, over="sequence", cu_seqlens=offsets))
        got += [v for v in kda.group_norm_bwd(x, 8, dy, weight=w, over="sequence", cu_seqlens=offsets).values() if v is not None]
    got.append(kda.group_norm_fwd(x, 1, weight=w))
    got += [v for v in kda.group_norm_bwd(x, 1, dy, weight=w).values() if v is not None]
    return got

graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    first = work()
for t in first:
    t.fill_(7)
graph.replay()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(first, work())), "not the bits of a call by itself"
print("the same")
"""


def test_first_calls_in_a_capture():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    run = subprocess.run([sys.executable, "-c", PROGRAM], capture_output=True, text=True, timeout=300, cwd=root,
                         env={**os.environ, "PYTHONPATH": root + os.pathsep + os.environ.get("PYTHONPATH", "")})
    assert run.returncode == 0 and run.stdout.strip() == "the same", run.stdout + run.stderr
