"""Outputs of the paged attention and the rotated append that lie in the memory
of what the call still reads, or in their own: refused, and what only looks so
is not.  No GPU is needed, no address is dereferenced."""
import pytest
import torch

import normalization_gemm_row_gb300 as pkg
from test_step_host import A, ARG, OTHER, append, attend, cache, moe, passes

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


# The cache of test_step_host: 10 pages of 16 tokens of 2 heads of 64; a page is 2048 elements.
@pytest.mark.parametrize("kw", [
    dict(k_page_stride=1024), dict(v_page_stride=2047 - 63), dict(v_page_stride=64), dict(k_token_stride=64), dict(v_token_stride=96),
    dict(k_page_stride=128, k_token_stride=128 * 9),                    # pages inside tokens, of too few
    dict(v=A), dict(v=A + 128), dict(v=A + 10 * 2048 * 2 - 16), dict(v=A - 64),
    dict(k_page_stride=4096, v_page_stride=4096, v=A + 2048),           # v's pages half over k's
    dict(k_head_stride=128, v_head_stride=128, k_token_stride=256, v_token_stride=256, k_page_stride=4096, v_page_stride=4096, v=A + 256)])
def test_append_refuses_caches_with_shared_places(kw):
    assert append(cache(**kw)) == ARG


@host_only
@pytest.mark.parametrize("kw", [
    dict(v=A + 10 * 2048 * 2), dict(k_page_stride=2048 + 8),
    dict(k_page_stride=4096, v_page_stride=4096, v=A + 2048 * 2),       # [pages, 2, tokens, heads, dim]
    dict(k_token_stride=256, v_token_stride=256, k_page_stride=4096, v_page_stride=4096, v=A + 256),     # [pages, tokens, 2, ...]
    dict(k_head_stride=128, v_head_stride=128, k_token_stride=256, v_token_stride=256, k_page_stride=4096, v_page_stride=4096, v=A + 128),
    dict(k_head_stride=1024, k_token_stride=64, k_page_stride=4096, v_page_stride=4096, v=A + 2048 * 2),  # k by heads, v by tokens
    dict(k_token_stride=144, k_head_stride=72, k_page_stride=4352, v_page_stride=4352, v=A + 2304 * 2),   # k padded, in one page
    dict(k_page_stride=128, k_token_stride=128 * 10),                   # pages inside tokens
    dict(pages=1, k_page_stride=1), dict(page_size=1, k_token_stride=1, v_token_stride=0)])
def test_append_takes_caches_whose_places_are_apart(kw):
    assert passes(append(cache(**kw)))


@pytest.mark.parametrize("kw", [
    dict(q_out_token=511), dict(q_out_token=64), dict(q_out_token=1), dict(q_out_head=96, q_out_token=512), dict(q_out_head=200, q_out_token=64),
    dict(q=OTHER + 2), dict(q=OTHER - 4 * ROW + 2), dict(q=OTHER + 16, q_token=512), dict(k=OTHER), dict(v=OTHER + 4 * ROW - 2),
    dict(q=OTHER - HEAD, q_token=640, q_out_token=640)])
def test_append_refuses_rotated_queries_over_inputs_or_themselves(kw):
    assert append(**kw) == ARG


@host_only
@pytest.mark.parametrize("kw", [
    dict(q=OTHER), dict(q=OTHER + 4 * ROW), dict(k=OTHER - 4 * 2 * HEAD), dict(q_out_head=256, q_out_token=64),
    dict(T=1, q_out_token=1), dict(T=1, H=1, q_out_head=1),
    # parts of rows of 2048: q, then q_out, k and v behind them
    dict(q=FAR, q_token=2048, q_out=FAR + ROW, q_out_token=2048, k=FAR + 2 * ROW, k_token=2048, v=FAR + 2 * ROW + 2 * HEAD, v_token=2048),
    # heads of q and of q_out in turn
    dict(q=FAR, q_head=128, q_token=1024, q_out=FAR + HEAD, q_out_head=128, q_out_token=1024)])
def test_append_takes_rotated_queries_apart(kw):
    assert passes(append(**kw))


# The experts' layer of test_step_host: 4 tokens of 64 elements (512 bytes), 2 choices each (32 bytes).
@pytest.mark.parametrize("kw", [
    dict(experts=A), dict(weights=A), dict(experts=A + 508), dict(weights=A - 28), dict(y=OTHER, experts=OTHER + 4),
    dict(y=OTHER, weights=OTHER), dict(y=OTHER, experts=A + 4), dict(experts=OTHER, weights=OTHER), dict(experts=OTHER, weights=OTHER + 28)])
def test_experts_refuse_a_choice_over_rows_or_weights(kw):
    assert moe(**kw) == ARG


@host_only
@pytest.mark.parametrize("kw", [
    dict(experts=A + 512), dict(weights=A - 32), dict(experts=OTHER, weights=OTHER + 32), dict(weights=OTHER), dict(y=A + 16, experts=OTHER)])
def test_experts_take_a_choice_apart(kw):
    assert passes(moe(**kw))
