"""The kernel timing of the linear cross entropy's calls: each launch counts,
the copy of W at widths that are no multiple of 8 among them."""
import pytest
import torch

import normalization_gemm_row_gb300 as ngr
from normalization_gemm_row_gb300 import binding as B
import ce_reference as C

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("K,M,kernels", [
    (64, 200, 3),       # gather (with the tokens' index), z, loss
    (61, 200, 4),       # W's copy first
    (64, 1500, 4)])     # the index apart
def test_launches_of_the_loss(K, M, kernels):
    ngr.build()
    d = {k: v.cuda() for k, v in C.case(M, K, 700, torch.bfloat16, seed=K).items()}
    ngr.fused_linear_cross_entropy(d["x"], d["W"], d["target"])
    B.kernel_timing_start(2)
    for _ in range(2):
        ngr.fused_linear_cross_entropy(d["x"], d["W"], d["target"])
    torch.cuda.synchronize()
    calls = B.kernel_timing_stop()
    assert [len(c) for c in calls] == [kernels] * 2
    assert all(ms > 0 for c in calls for ms in c)


def test_copy_comes_first_in_the_gradient():
    """The timing keeps a call's first kernels: the copy of a large W is the
    longest of them where there is one token."""
    ngr.build()
    d = {k: v.cuda() for k, v in C.case(1, 1001, 60000, torch.bfloat16, seed=1).items()}
    _, lse = ngr.fused_linear_cross_entropy(d["x"], d["W"], d["target"])
    args = (d["dloss"], lse, d["x"], d["W"], d["target"])
    ngr.fused_linear_cross_entropy_backward(*args)
    B.kernel_timing_start(1)
    ngr.fused_linear_cross_entropy_backward(*args)
    torch.cuda.synchronize()
    copy, gather, *_ = B.kernel_timing_stop()[0]
    assert copy > 4 * gather
