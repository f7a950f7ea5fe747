"""Refusals of the block join's and the cross entropy's helpers that need no
GPU, beside those of the entry points' own files."""
import pytest
import torch

import normalization_gemm_row_gb300 as pkg
from normalization_gemm_row_gb300 import binding as B

A, OTHER, WS = 0x10000, 0x20000, 0x100000      # fake addresses: never dereferenced


@pytest.fixture(scope="module", autouse=True)
def _lib():
    pkg.build()


def forward(h, y, norm2=2, M=4):
    return B.ngr_fused_norm_gate_residual_norm(2, norm2, A, A, None, 0, A, None, A, None, 1e-5, 1e-5, 1.0, 1.0, M, 64, 0, h, y,
                                               None, None)


def backward(dx, dr, M=4):
    return B.ngr_fused_norm_gate_residual_norm_backward(2, 2, A, A, A, A, None, 0, A, None, A, A, 1.0, 1.0, M, 64, 0, dx, dr,
                                                        None, None, None, None, None, WS, 1 << 20, None)


def test_two_outputs_in_one_memory():
    assert forward(A, A) == -9
    assert backward(A, A) == -9
    # (one device check later: no GPU, or outputs that differ)
    if not torch.cuda.is_available():
        for rc in (forward(A, OTHER), forward(A, A, norm2=0), backward(A, OTHER), backward(A, None)):
            assert rc in (-6, -7)
    assert forward(A, A, M=0) == 0


def test_workspace_to_ask():
    with pytest.raises(ValueError, match="CUDA"):
        pkg.check_workspace(torch.zeros(256, dtype=torch.uint8))
