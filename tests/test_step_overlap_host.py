"""Outputs of the paged attention and the rotated append that lie in the memory
of what the call still reads, or in their own: refused, and what only looks so
is not.  No GPU is needed, no address is dereferenced."""
import pytest
import torch

import normalization_gemm_row_gb300 as pkg
from test_step_host import A, ARG, OTHER, append, attend, cache, passes

FAR = 0x40000000


@pytest.fixture(scope="module", autouse=True)
def _lib():
    pkg.build()


host_only = pytest.mark.skipif(torch.cuda.is_available(), reason="fake addresses must not reach a device")
ROW, HEAD = 8 * 64 * 2, 64 * 2      # bytes of a dense row of 8 heads of 64, and of a head


@pytest.mark.parametrize("kw", [
    dict(q_row=1024), dict(q_row=640),                                  # q's rows wider than out's, from one address
    dict(q_row=64, q_head=256),                                         # heads first
    dict(out=A + HEAD), dict(out=A + 16), dict(out=A - 16), dict(out=A + 3 * ROW), dict(out=A - 4 * ROW + 16),
    dict(q_row=0),                                                      # one row for all
    dict(q_row=1024, out=A + 512 * 2),                                  # in the gap behind q's first row, and over its second
    dict(lse=A), dict(lse=A + 4 * ROW - 4), dict(lse=A - 4),
    dict(out=OTHER, lse=OTHER + 64), dict(out=OTHER, lse=OTHER - 4)])
def test_attention_refuses_outputs_over_queries(kw):
    assert attend(**kw) == ARG


@host_only
@pytest.mark.parametrize("kw", [
    dict(), dict(out=A + 4 * ROW), dict(out=A - 4 * ROW), dict(lse=A + 4 * ROW), dict(lse=A - 4 * 8 * 4),
    dict(B=1, q_row=7), dict(B=1, H=2, G=2, q_row=7),
    dict(q_row=4096, out=A + 512 * 2 * 2, B=3, H=8),                     # out within the gap behind q's first row
    dict(q_row=640, out=A + 3 * 640 * 2 + ROW)])
def test_attention_takes_outputs_apart_from_queries(kw):
    assert passes(attend(**kw))
