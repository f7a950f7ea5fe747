"""A target outside the vocabulary, as a user of the tensor helpers learns of
it: by asking the workspace, or at once with NGR_DEBUG=1."""
import os
import subprocess
import sys

import pytest
import torch

import normalization_gemm_row_gb300 as ngr
from normalization_gemm_row_gb300 import binding as B
import ce_reference as C

pytestmark = pytest.mark.gpu


def test_asking_the_workspace():
    ngr.build()
    M, K, V = 40, 64, 90
    d = {k: v.cuda() for k, v in C.case(M, K, V, torch.float16, seed=1).items()}
    ws = [torch.empty(B.ngr_linear_cross_entropy_workspace_bytes(i, M, K, V), dtype=torch.uint8, device="cuda") for i in (0, 1)]
    args = (d["x"], d["W"], d["target"])
    _, lse = ngr.fused_linear_cross_entropy(*args, workspace=ws[0])
    ngr.fused_linear_cross_entropy_backward(d["dloss"], lse, *args, workspace=ws[1])
    for w in ws:
        ngr.check_workspace(w)
    d["target"][3] = V
    loss, lse = ngr.fused_linear_cross_entropy(*args, workspace=ws[0])
    dx, _ = ngr.fused_linear_cross_entropy_backward(d["dloss"], lse, *args, workspace=ws[1])
    for w in ws:
        with pytest.raises(ngr.NgrError) as e:
            ngr.check_workspace(w, torch.cuda.current_stream())
        assert e.value.status == -9
        ngr.check_workspace(w)      # once
    assert loss[3] == 0 and lse[3] == 0 and (dx[3] == 0).all()


CHILD = r"""
import torch
import normalization_gemm_row_gb300 as ngr
x, W = torch.randn(9, 64, device="cuda").half(), torch.randn(50, 64, device="cuda").half()
t = torch.arange(9, device="cuda")
def both():
    loss, lse = ngr.fused_linear_cross_entropy(x, W, t)
    ngr.fused_linear_cross_entropy_backward(loss, lse, x, W, t)
both()
print("fine")
t[4] = 50
for call in (lambda: ngr.fused_linear_cross_entropy(x, W, t),
             lambda: ngr.fused_linear_cross_entropy_backward(t.float(), t.float(), x, W, t)):
    try:
        call()
    except ngr.NgrError as e:
        print("raised", e.status)
"""


def test_raised_with_debug():
    env = dict(os.environ, NGR_DEBUG="1")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    p = subprocess.run([sys.executable, "-c", CHILD], cwd=root, env=env, capture_output=True, text=True, timeout=300)
    assert p.returncode == 0, p.stderr
    assert p.stdout.split("\n")[:3] == ["fine", "raised -9", "raised -9"], p.stdout
