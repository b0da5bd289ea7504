"""The first call of each operator in a process may be a captured one: nothing it sets up is refused by a capture."""
import subprocess
import sys

import pytest

from gpu_util import need_gpu

pytestmark = pytest.mark.gpu

SCRIPT = """
import os, sys
sys.path[:0] = [os.getcwd(), os.path.join(os.getcwd(), "tests")]
import torch, verify_weight_streaming_b200 as mr, w4_util
w = w4_util.weight(1, (), 96, 256, 64, True)
packed, fmt = w4_util.pack(mr, w)
a = torch.ones((2, 256), dtype=torch.bfloat16, device="cuda")
c = torch.zeros((2, 96), device="cuda")
up = torch.ones((3, 64, 256), dtype=torch.bfloat16, device="cuda") / 64
down = torch.ones((3, 256, 32), dtype=torch.bfloat16, device="cuda")
ids = torch.tensor([[0, 2], [1, -1]], dtype=torch.int32, device="cuda")
wts = torch.ones((2, 2), device="cuda")
y = torch.zeros((2, 256), device="cuda")
ws = torch.zeros(mr.moe_window_workspace_bytes(2, 2, 256, 32), dtype=torch.uint8, device="cuda")
lse = torch.zeros(2, device="cuda")
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    mr.mrgemv_w4(a, packed, c, fmt)
    mr.moe_window_bf16(a, ids, wts, up, down, y, ws)
    mr.token_logprobs(c, lse=lse)
graph.replay()
torch.cuda.synchronize()
assert abs(c - torch.from_numpy(w4_util.dense64(w).sum(1)).cuda()).max() < 1e-3
h = 4.0 / (1 + torch.exp(torch.tensor(-4.0))) * 4.0 * 32
assert abs(y[0] - 2 * h).max() < 1e-3 * h and abs(y[1] - h).max() < 1e-3 * h
assert abs(lse - torch.logsumexp(c, 1)).max() < 1e-4
assert mr.mr_poll_errors() == 0
print("ok")
"""


def test_first_call_in_capture():
    need_gpu()
    run = subprocess.run([sys.executable, "-c", SCRIPT], capture_output=True, text=True, timeout=300)
    assert run.returncode == 0 and run.stdout.strip().endswith("ok"), run.stdout + run.stderr
