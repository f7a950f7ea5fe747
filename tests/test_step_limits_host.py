"""The paged attention at the limits of its sizes and scale: the last that is
taken and the first that is refused.  No GPU is needed, no address is
dereferenced."""
import pytest
import torch

import normalization_gemm_row_gb300 as pkg
from test_step_host import ARG, SHAPE, attend, cache, passes

UNITS = 1 << 32      # 16-byte units of 64 GiB


@pytest.fixture(scope="module", autouse=True)
def _lib():
    pkg.build()


def reaching(last, D, which):
    """A cache whose last head starts `last` 16-byte units behind its first: pages of 2 tokens, and one step that is odd
    enough to hit the number."""
    tokens = 2 * D
    page = 2 * tokens
    pages = last * 8 // page                                     # of these, then a last token further off
    far = last * 8 - (pages - 1) * page - D                      # step of the page's second token: what is left
    f = {f"{which}_page_stride": page, f"{which}_token_stride": far, f"{which}_head_stride": D}
    other = "v" if which == "k" else "k"
    f.update({f"{other}_page_stride": 0, f"{other}_token_stride": D * 2, f"{other}_head_stride": D})
    assert (pages - 1) * page + far + D == last * 8 and far % 8 == 0
    return cache(pages=pages, page_size=2, **f)


def call(c, D):
    return attend(c, D=D, q_row=8 * D, q_head=D)


@pytest.mark.parametrize("which", ["k", "v"])
@pytest.mark.parametrize("D", [16, 64, 80, 96, 128, 192, 256])
def test_a_cache_reaches_over_64_gib_and_no_further(which, D):
    if not torch.cuda.is_available():      # (fake addresses must not reach a device)
        assert passes(call(reaching(UNITS - D // 8, D, which), D))
    for past in (1, 2, D // 8 - 1, D // 8, D // 8 + 1):
        assert call(reaching(UNITS - D // 8 + past, D, which), D) == SHAPE


def test_the_smallest_heads_end_a_unit_earlier():
    """(a head of one unit: the largest number stands for none)"""
    if not torch.cuda.is_available():
        assert passes(call(reaching(UNITS - 2, 8, "k"), 8))
    assert call(reaching(UNITS - 1, 8, "k"), 8) == SHAPE


@pytest.mark.parametrize("sign", [1, -1])
def test_scales_whose_exponents_of_2_pass_fp32(sign):
    """(the kernels' exponentials are of 2: times log2 e, such a scale would be infinite)"""
    assert attend(scale=sign * 3e38) == ARG and attend(scale=sign * float("inf")) == ARG
    if not torch.cuda.is_available():
        assert passes(attend(scale=sign * 2.0 ** 127)) and passes(attend(scale=sign * 1e-45)) and passes(attend(scale=0.0))
