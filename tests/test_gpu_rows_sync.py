"""What tq_sync costs: it asks the GPU for the given-up waits of the row
products' formats that this process has launched, and of no others."""
import os
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CODE = """
import sys
sys.path[:0] = [{root!r}, {tests!r}]
import torch
from torch.profiler import ProfilerActivity, profile
import group_scale_search_b200 as tq
import rows_ref as ref

def copies():
    tq.tq_sync()
    with profile(activities=[ProfilerActivity.CUDA, ProfilerActivity.CPU]) as p:
        tq.tq_sync()
    return sum(e.count for e in p.key_averages() if "Memcpy DtoH" in e.key)

x = torch.ones(100, 64, dtype=torch.bfloat16, device="cuda")
found = [copies()]
for fmt in ("int3", "nvfp4"):
    w = ref.Weights(fmt, 1, 80, 64, 1, "cuda").handle(tq)
    tq.tq_dequant_matmul(x[:3], w)    # (the few-token kernel waits for nothing)
    tq.tq_dequant_matmul(x, w)
    found.append(copies())
print("copies", *found)
"""


def test_tq_sync_asks_for_what_was_launched():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    code = CODE.format(root=ROOT, tests=os.path.join(ROOT, "tests"))
    out = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert out.returncode == 0, out.stderr[-2000:]
    before, one, two = map(int, out.stdout.split("copies")[-1].split())
    assert before > 0   # (the other pipelines' counters: the profiler sees them)
    assert (one - before, two - before) == (1, 2)
