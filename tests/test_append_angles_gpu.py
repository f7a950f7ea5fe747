"""Rotations by frequencies from one end of FP32's range to the other."""
from fractions import Fraction

import pytest
import torch

import normalization_gemm_row_gb300 as ngr
import kv_reference as R

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
PI = Fraction(3141592653589793238462643383279502884197169399375105820974944592307816406286208998628034825342117067982148086513282306647093844609550582231,
              10 ** 138)


@pytest.fixture(scope="module", autouse=True)
def _built():
    ngr.build()
    torch.cuda.init()


def angles(positions, inv):
    """position x inv modulo 2 pi, in rationals."""
    out = torch.zeros((len(positions), len(inv)), dtype=torch.float64)
    for t, p in enumerate(positions):
        for i, f in enumerate(inv):
            x = Fraction(f) * p
            out[t, i] = float(x - 2 * PI * (x / (2 * PI)).__floor__())
    return out


@pytest.mark.parametrize("low,high", [(0, 40), (40, 64), (64, 88), (88, 128), (-40, 0), (-149, -40)])
def test_frequencies_by_their_exponent(low, high):
    g = R.generator(high + 200)
    n, D = 64, 128
    m = 1 + torch.rand(n, generator=g, dtype=torch.float64)
    e = low + (high - low) * torch.rand(n, generator=g, dtype=torch.float64)
    inv = (m * torch.exp2(e.floor())).float()
    inv[0] = 2.0 ** low
    inv[1] = torch.finfo(torch.float32).max if high == 128 else 2.0 ** (high - 1) * (2 - 2.0 ** -23)
    inv[1::2] *= -1
    assert torch.isfinite(inv).all()
    positions = [1, 2, 3, 4097, 123456789, (1 << 31) - 1]
    q = torch.randn((len(positions), 1, D), generator=g).to(BF16)
    size = 1 << 16
    table = torch.zeros((len(positions), ((1 << 31) - 1) // size + 1), dtype=torch.int32)
    kc, vc = (torch.zeros((1, size, 1, D), dtype=BF16, device="cuda") for _ in range(2))
    got = ngr.fused_rope_append_kv(q.cuda(), q.cuda(), q.cuda(), kc, vc, table.cuda(),
                                   torch.tensor(positions, dtype=torch.int32, device="cuda"), inv_freq=inv.cuda())
    angle = angles(positions, inv.tolist())[:, None]
    c, s = torch.cos(angle), torch.sin(angle)
    a, b = q.double()[..., :n], q.double()[..., n:]
    R.check_rotated(got, torch.cat((a * c - b * s, a * s + b * c), -1), torch.cat((a.abs() + b.abs(),) * 2, -1), BF16, f"2^{low} to 2^{high}")


def test_frequencies_that_are_not_finite():
    inv = torch.tensor([float("inf"), -float("inf"), float("nan"), 1.0])
    q = torch.ones((1, 1, 8), dtype=BF16, device="cuda")
    kc, vc = (torch.zeros((1, 8, 1, 8), dtype=BF16, device="cuda") for _ in range(2))
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = ngr.fused_rope_append_kv(q, q, q, kc, vc, zero[:, None], zero + 3, inv_freq=inv.cuda())[0, 0].cpu()
    assert torch.isnan(got).tolist() == [True, True, True, False] * 2
