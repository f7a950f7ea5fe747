"""Block tables with every number that is no page, in both forms of the paged
attention: their tokens are left out, and the call reports it."""
import pytest
import torch

import normalization_gemm_row_gb300 as ngr
import kv_reference as R
from test_attend_gpu import call, data

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _built():
    ngr.build()
    torch.cuda.init()


@pytest.mark.parametrize("entry", [-(1 << 31), -(1 << 31) + 1, -1, "pages", (1 << 31) - 1])
@pytest.mark.parametrize("B,page_size", [(3, 16), (3, 1), (200, 16), (200, 1)])      # a CTA an item; runs
@pytest.mark.parametrize("where", ["first", "middle", "last", "all"])
def test_entries_that_are_no_pages(entry, B, page_size, where):
    lengths = [40 + b % 150 for b in range(B)]
    d = data(lengths, 4, 1, 64, page_size, BF16, dirty=False, seed=B)
    row = B // 2
    last = (lengths[row] - 1) // page_size
    at = {"first": [0], "middle": [last // 2], "last": [last], "all": list(range(last + 1))}[where]
    d["table"][row, at] = d["k"].shape[0] if entry == "pages" else entry
    n = ngr.binding.ngr_paged_attention_workspace_bytes(B, 4, 1, 64, d["table"].shape[1] * page_size, 0)
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
    out, lse = call(d, workspace=ws)
    R.check_attention(out, lse, R.attention(d["q"], d["k"], d["v"], d["table"], d["lengths"], 0.125))
    with pytest.raises(ngr.NgrError) as e:
        ngr.check_workspace(ws)
    assert e.value.status == -9
    # where no token's page is, anything may stand
    d = data(lengths, 4, 1, 64, page_size, BF16, dirty=False, seed=B)
    d["table"][row, last + 1:] = 7 if entry == "pages" else entry
    call(d, workspace=ws)
    ngr.check_workspace(ws)
