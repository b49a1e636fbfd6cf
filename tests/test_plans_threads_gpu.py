"""Handles made and used by several threads of a process that has none yet."""
import os
import subprocess
import sys

import pytest
import torch

from ssm_sequence_layer_gb300 import build

pytestmark = pytest.mark.gpu

PROGRAM = """
import threading
import torch
from ssm_sequence_layer_gb300 import binding as B

g = torch.Generator().manual_seed(0)
M, N, K = 3000, 520, 264
x, W, dy = (torch.randn(*s, generator=g).to(torch.bfloat16).cuda() for s in ((M, K), (N, K), (M, N)))
torch.cuda.synchronize()
start, results = threading.Barrier(8), [None] * 8

def work(i):
    start.wait()
    with B.Tokens(M, 64, 64) as t, torch.cuda.stream(torch.cuda.Stream()):
        out = t.linear(x, W)["y"], t.linear_backward(dy, W), t.linear_weight_backward(dy, x)["dW"]
        torch.cuda.current_stream().synchronize()
        t.last_device_status()
    results[i] = out

threads = [threading.Thread(target=work, args=(i,)) for i in range(8)]
for t in threads: t.start()
for t in threads: t.join()
assert all(r is not None and all(torch.equal(a, b) for a, b in zip(r, results[0])) for r in results)
print("equal")
"""


def test_first_handles_of_several_threads():
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", PROGRAM], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "equal", r.stderr[-2000:]
