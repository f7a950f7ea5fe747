"""NGR_TRACE=1: the calls of a model's tail print the kernel variants they
chose, as the layers do."""
import os
import re
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

CHILD = r"""
import torch
import normalization_gemm_row_gb300 as ngr
x, W = torch.randn(40, 520, device="cuda").half(), torch.randn(300, 520, device="cuda").half()
g, t = torch.ones(520, device="cuda").half(), torch.arange(40, device="cuda")
h, y, st = ngr.fused_norm_gate_residual_norm(x, x, gamma1=g, gamma2=g, return_stats=True)
ngr.fused_norm_gate_residual_norm_backward(y, h, x, x, st, gamma1=g, gamma2=g)
loss, lse = ngr.fused_linear_cross_entropy(x, W, t)
ngr.fused_linear_cross_entropy_backward(loss, lse, x, W, t)
ngr.fused_rmsnorm_linear(x, g, W)
torch.cuda.synchronize()
"""
LINES = [r"ngr: block join M=40 N=520 norms=2,2 aligned cluster=1 cols=520 threads=\d+ x \d+ vecs=\d+ grid=\d+",
         r"ngr: block join gradient M=40 N=520 norms=2,2 aligned cluster=1 cols=520 threads=\d+ x \d+ vecs=\d+ grid=\d+",
         r"ngr: cross entropy z: 300 columns, width=\d+ splits=1 grid=\d+",
         r"ngr: cross entropy dz: 300 columns, width=\d+ splits=1 grid=\d+",
         r"ngr: cross entropy dx: 520 columns, width=256 splits=\d+ grid=\d+",
         r"ngr: cross entropy dW: 520 columns, width=256 splits=1 grid=\d+",
         r"ngr: tile kernel M=40 .*"]


def test_variants_are_printed():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    for on, lines in (("1", LINES), ("0", [])):
        p = subprocess.run([sys.executable, "-c", CHILD], cwd=root, env=dict(os.environ, NGR_TRACE=on), capture_output=True,
                           text=True, timeout=300)
        assert p.returncode == 0, p.stderr
        got = [line for line in p.stderr.split("\n") if line.startswith("ngr: ")]
        assert len(got) == len(lines), p.stderr
        for a, b in zip(got, lines):
            assert re.fullmatch(b, a), (a, b)
