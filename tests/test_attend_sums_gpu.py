"""Long sums of the paged attention: batches whose rows are a warp's own for
thousands of tiles."""
import pytest
import torch

import normalization_gemm_row_gb300 as ngr
import kv_reference as R

pytestmark = pytest.mark.gpu
F16 = torch.float16


@pytest.fixture(scope="module", autouse=True)
def _built():
    ngr.build()
    torch.cuda.init()


@pytest.mark.parametrize("rows,n,H,G,D", [(256, 131072, 8, 8, 128), (256, 131072, 16, 8, 64), (64, 131072, 144, 8, 256), (300, 100000, 8, 8, 80)])
def test_sums_do_not_drift(rows, n, H, G, D):
    """Equal scores: every output is a plain mean of values (of one sign).  Pages repeat."""
    page, pages = 64, 16
    g = R.generator(D)
    k = torch.zeros((pages, page, G, D), dtype=F16)
    v = (0.75 + 0.75 * torch.rand((pages, page, G, D), generator=g)).to(F16)
    q = torch.randn((rows, H, D), generator=g).to(F16)
    table = (torch.arange(-(-n // page), dtype=torch.int32) % pages).repeat(rows, 1).cuda()
    lengths = torch.full((rows,), n, dtype=torch.int32, device="cuda")
    out = ngr.fused_paged_attention(q.cuda(), k.cuda(), v.cuda(), table, lengths).double().cpu()
    at = torch.arange(n) % (page * pages)
    times = torch.bincount(at, minlength=page * pages).double()
    want = torch.einsum("n,ngd->gd", times, v.double().view(-1, G, D)) / n
    want = want.repeat_interleave(H // G, dim=0)
    # the weights are 1 exactly; a tile's 16 values are added to within 2^-22, and n / 16 tiles by additions of half a step
    # 2^-24 of what is there so far, on average half of all; then the output's rounding
    tol = (n / 16 * 2.0 ** -25 + 2.0 ** -22 + 64 * 2.0 ** -24 + R.U[F16]) * want
    r = ((out - want).abs() / tol).max().item()
    assert r <= 1, f"worst {r:.2f} times the tolerance"
