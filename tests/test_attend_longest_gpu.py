"""Paged attention over as many tokens as a length can count: 2^31 - 1, in pages
that a row of the table repeats."""
import pytest
import torch

import normalization_gemm_row_gb300 as ngr
import kv_reference as R

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
PAGE, D, H = 1 << 20, 8, 2
MOST = (1 << 31) - 1


@pytest.fixture(scope="module", autouse=True)
def _built():
    ngr.build()
    torch.cuda.init()


def check(lengths):
    g = R.generator(11)
    k = torch.randn((1, PAGE, 1, D), generator=g).to(BF16)
    v = (1 + 0.5 * torch.randn((1, PAGE, 1, D), generator=g)).to(BF16)
    q = torch.randn((len(lengths), H, D), generator=g).to(BF16)
    table = torch.zeros((len(lengths), (MOST + 1) // PAGE), dtype=torch.int32, device="cuda")
    n = torch.tensor(lengths, dtype=torch.int32)
    size = ngr.binding.ngr_paged_attention_workspace_bytes(len(lengths), H, 1, D, table.shape[1] * PAGE, 0)
    ws = torch.full((size,), 255, dtype=torch.uint8, device="cuda")
    out, lse = ngr.fused_paged_attention(q.cuda(), k.cuda(), v.cuda(), table, n.cuda(), return_lse=True, workspace=ws)
    ngr.check_workspace(ws)
    out, lse = out.double().cpu(), lse.double().cpu()
    at, scale = torch.arange(PAGE), D ** -0.5
    kd, vd = k[0, :, 0].double(), v[0, :, 0].double()
    for b in sorted({0, 1, 2, len(lengths) - 1}):
        times = (lengths[b] // PAGE + (at < lengths[b] % PAGE)).double()[:, None]      # a slot's tokens
        z = kd @ q[b].double().t() * scale
        size_z = kd.abs() @ q[b].double().abs().t() * scale
        e = times * torch.exp(z)
        want, want_lse = (e / e.sum(0)).t() @ vd, torch.log(e.sum(0))
        # as in kv_reference.py: scores; 2432 workers' sums, 16 tokens at a time, and their joining
        dz = ((D / 16 + 24) * 2.0 ** -23 * size_z + 2.0 ** -20).max()
        chain = (lengths[b] / 16 / 2432 + 2432 + 64) * 2.0 ** -23
        tol = (2 * dz + R.U[BF16] ** 2 + chain) * ((e / e.sum(0)).t() @ vd.abs()) + R.U[BF16] * want.abs()
        assert ((out[b] - want).abs() <= tol).all(), (b, lengths[b])
        assert ((lse[b] - want_lse).abs() <= 2 * dz + chain + 2.0 ** -22 * want_lse.abs()).all(), (b, lengths[b])


def test_lengths_up_to_the_most_that_32_bits_hold():
    check([MOST, 5, MOST - 15, MOST - 14, 0, 17])


def test_the_longest_row_among_more_rows_than_the_device_has_warps():
    check([3, MOST, 40] + [2] * 2500)
