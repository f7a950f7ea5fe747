"""With NGR_DEBUG=1 the join's gradient reads its workspace's error word, as
every call does that waits inside a kernel.  The word is set here as a wait
that ran out would leave it: by a graph of small fills on another stream that
runs on while the gradient does (which clears it first)."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

CHILD = r"""
import torch
import normalization_gemm_row_gb300 as ngr
from normalization_gemm_row_gb300 import binding as B
M = N = 2048
x, r, dy, dh = (torch.randn(M, N, device="cuda").half() for _ in range(4))
v = torch.ones(N, device="cuda").half()
kw = dict(norm1=1, gamma1=v, beta1=v, norm2=1, gamma2=v, beta2=v)
h, y, st = ngr.fused_norm_gate_residual_norm(x, r, return_stats=True, **kw)
ws = torch.zeros(B.ngr_norm_gate_residual_norm_workspace_bytes(1, 1, 0, M, N), dtype=torch.uint8, device="cuda")
word = ws[:4].view(torch.int32)
def gradient():
    ngr.fused_norm_gate_residual_norm_backward(dy, dh, x, r, st, workspace=ws, **kw)
    torch.cuda.synchronize()
gradient()
other, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    for _ in range(4000):
        word.fill_(1)
torch.cuda.synchronize()
with torch.cuda.stream(other):
    graph.replay()
try:
    gradient()
    print("nothing reported")
except ngr.NgrError as e:
    print("reported", e.status)
torch.cuda.synchronize()
gradient()
print("clean", int(word.item()))
"""


def test_error_word_is_read():
    env = dict(os.environ, NGR_DEBUG="1")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    p = subprocess.run([sys.executable, "-c", CHILD], cwd=root, env=env, capture_output=True, text=True, timeout=300)
    assert p.returncode == 0, p.stderr
    assert p.stdout.split("\n")[:2] == ["reported -8", "clean 0"], p.stdout
