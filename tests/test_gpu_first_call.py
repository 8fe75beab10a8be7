"""A process whose first call of the library is captured into a graph (one fresh process per call)."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = """
import sys
sys.path[:0] = [{root!r}, {tests!r}]
import torch
import weight_only_quantization_awq_b200 as awq
from test_gpu_train import ce_case, packed, rand
w, _, _ = packed(640, 256, 64, True, True, 1)
wl, _, _ = packed(192, 256, 64, False, True, 2)
M = {M}
x, dh, dy = rand(M, 256, 3), rand(M, 320, 4), rand(M, 192, 5)
xc, W, labels = ce_case(M, 999, 128, 6)
lse, dloss = torch.full((M,), 9.0, device="cuda"), torch.ones(M, device="cuda")
call = {{"gated": lambda: (awq.awq_gated_w4a16(x, *w, group_size=64),),
        "gated_grad": lambda: (awq.awq_gated_w4a16_grad(dh, x, *w, group_size=64),),
        "linear": lambda: (awq.awq_linear_w4a16(x, *wl, group_size=64),),
        "linear_grad": lambda: (awq.awq_linear_w4a16_grad(dy, *wl, group_size=64),),
        "ce": lambda: awq.awq_cross_entropy(xc, W, labels),
        "ce_grad": lambda: awq.awq_cross_entropy_grad(xc, W, labels, lse, dloss)}}[{name!r}]
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    outs = call()
for t in outs:
    t.fill_(float("nan"))
g.replay()
torch.cuda.synchronize()
for a, b in zip(outs, call()):
    assert torch.equal(a, b)
print("same")
"""


@pytest.mark.parametrize("name,M", [("gated", 2), ("gated", 400), ("gated_grad", 40), ("linear", 3), ("ce", 300),
                                    ("ce_grad", 70)])
def test_first_call_captured(name, M):
    code = PROGRAM.format(root=ROOT, tests=os.path.join(ROOT, "tests"), name=name, M=M)
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip().endswith("same"), r.stderr[-2000:]
