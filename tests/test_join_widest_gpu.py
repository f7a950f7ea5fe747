"""The block join's gradient at the widest rows, where shifted rows and rows
with five column sums (LayerNorm on both sides, a gate row for fewer than 16
tokens) take clusters of 16 CTAs."""
import pytest
import torch

import normalization_gemm_row_gb300 as ngr
import join_reference as R
import test_join_gpu as J

pytestmark = pytest.mark.gpu
LAYER, RMS = J.LAYER, J.RMS


@pytest.fixture(scope="module", autouse=True)
def _built():
    ngr.build()
    torch.cuda.init()


@pytest.mark.parametrize("N", [65472, 65473, 65530, 65535])
def test_shifted_rows(N):
    for norm1, norm2, gates, dtype in ((LAYER, LAYER, 1, torch.float16), (RMS, RMS, 0, torch.bfloat16)):
        d = R.case(3, N, norm1, norm2, gates, dtype, seed=N)
        J.compare(d, norm1, norm2, f"{N} {norm1}{norm2}")


@pytest.mark.parametrize("M,N,gates", [(2, 61440, 2), (4, 61448, 4), (6, 65536, 2), (2, 65536, 2), (2, 61313, 2), (4, 65535, 2)])
def test_five_sums(M, N, gates):
    d = R.case(M, N, LAYER, LAYER, gates, torch.bfloat16, seed=M + N)
    J.compare(d, LAYER, LAYER, f"{M}x{N}, {gates} gates", s=0.5)


def test_many_rows_of_a_wide_cluster():
    """More rows than clusters run at once."""
    d = R.case(40, 65535, RMS, RMS, 1, torch.bfloat16, seed=1)
    J.compare(d, RMS, RMS, "40 x 65535")


@pytest.mark.parametrize("offsets", [(1, 1, 1, 1), (0, 1, 2, 3)])
def test_one_element_off(offsets):
    """65536 columns whose rows start off a 16-byte boundary: all alike, and
    each array at a place of its own."""
    d = R.case(2, 65536, LAYER, LAYER, 2, torch.float16, seed=sum(offsets))
    c = J.cuda(d)
    for k, at in zip(("x", "residual", "dy", "dh"), offsets):
        c[k] = torch.empty(c[k].numel() + at, dtype=c[k].dtype, device="cuda")[at:].view(2, -1).copy_(c[k])
    args = J.how(c, LAYER, LAYER)
    h, y, st = ngr.fused_norm_gate_residual_norm(c["x"], c["residual"], return_stats=True, **args)
    got = {"h": h, "y": y}
    got.update(ngr.fused_norm_gate_residual_norm_backward(c["dy"], c["dh"], c["x"], c["residual"], st, **args))
    val, mag = R.reference(d, LAYER, LAYER)
    for k, v in val.items():
        R.check(got[k], v, mag[k], torch.float16, k)
