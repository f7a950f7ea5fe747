"""Gradient weights that are not finite: they concern their own token's dx,
and dW; every other token's dx keeps its precision."""
import pytest
import torch

import normalization_gemm_row_gb300 as ngr
import ce_reference as R

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("M", [60, 1100])       # (the tokens' index in the gather, and apart)
@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
def test_one_weight_that_is_not_finite(value, M, dtype):
    """A mean over many tokens: weights so small that fp16 needs its unit."""
    ngr.build()
    d = R.case(M, 64, 900, dtype, seed=3)
    # (the weights of W large, so that dx itself is inside fp16's range)
    d["dloss"] = torch.full((M,), 1.0 / 8192)
    d["W"], d["x"] = d["W"] * 64, d["x"] / 64
    bad = M // 3
    c = {k: v.cuda() for k, v in d.items()}
    c["dloss"][bad] = value
    _, lse = ngr.fused_linear_cross_entropy(c["x"], c["W"], c["target"])
    dx, dW = ngr.fused_linear_cross_entropy_backward(c["dloss"], lse, c["x"], c["W"], c["target"])
    good = torch.arange(M) != bad
    rest = {k: (v[good] if k != "W" else v) for k, v in d.items()}
    val, tol = R.reference(rest, 1.0, rest["dloss"])
    R.check(dx.cpu()[good], val["dx"], tol["dx"], "the other tokens' dx")
    assert not torch.isfinite(dx[bad]).any()
    assert not torch.isfinite(dW).any()
