"""The paged cache and the experts where offsets pass 31 bits: caches of 2.3e9
elements, expert weights of as many."""
import pytest
import torch

import normalization_gemm_row_gb300 as ngr
import kv_reference as K
import moe_reference as M

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _built():
    ngr.build()
    torch.cuda.init()


@pytest.mark.parametrize("layout", ["pages", "pages inside"])
def test_far_pages(layout):
    """Append to and attend over pages at both ends of a large cache."""
    page, G, D, H = 64, 8, 128, 16
    pages = 2300000000 // (page * G * D)
    shape = (pages, page, G, D) if layout == "pages" else (page, pages, G, D)
    kc, vc = (torch.empty(shape, dtype=BF16, device="cuda") for _ in range(2))
    if layout == "pages inside":
        kc, vc = kc.transpose(0, 1), vc.transpose(0, 1)
    near = [0, pages - 1, pages // 2, pages - 2, 7, pages - 3]
    table = torch.tensor([near[:3], near[3:]], dtype=torch.int32)
    g = K.generator(1)
    for p in near:
        kc[p].copy_(torch.randn((page, G, D), generator=g))
        vc[p].copy_(torch.randn((page, G, D), generator=g))
    q, k, v = (torch.randn((2, n, D), generator=g).to(BF16) for n in (H, G, G))
    positions = torch.tensor([2 * page + 5, page + 9], dtype=torch.int32)
    inv = (10000.0 ** (-torch.arange(0, D, 2, dtype=torch.float64) / D)).float()
    qr = ngr.fused_rope_append_kv(q.cuda(), k.cuda(), v.cuda(), kc, vc, table.cuda(), positions.cuda(), inv_freq=inv.cuda())
    lengths = positions + 1
    small = {n: torch.stack([t[p] for p in near]).cpu() for n, t in (("k", kc), ("v", vc))}
    for b, p in enumerate(positions.tolist()):
        at = 3 * b + p // page
        val, mag = K.rotate(k[b:b + 1].double(), positions[b:b + 1], inv, False)
        K.check_rotated(small["k"][at, p % page][None], val, mag, BF16, "k")
        assert torch.equal(small["v"][at, p % page], v[b])
    out, lse = ngr.fused_paged_attention(qr, kc, vc, table.cuda(), lengths.cuda(), return_lse=True)
    want = K.attention(qr.cpu(), small["k"], small["v"], torch.arange(6, dtype=torch.int32).view(2, 3), lengths, D ** -0.5)
    K.check_attention(out, lse, want)


def test_a_million_tokens():
    """One sequence whose tokens share a few pages: positions and tiles far beyond 16 bits."""
    page, n = 256, 1 << 20
    g = K.generator(2)
    kc, vc = (torch.randn((3, page, 1, 64), generator=g).to(F16) for _ in range(2))
    q = torch.randn((1, 4, 64), generator=g).to(F16)
    table = torch.tensor([[0, 1] * (n // page // 2)], dtype=torch.int32)
    out, lse = ngr.fused_paged_attention(q.cuda(), kc.cuda(), vc.cuda(), table.cuda(), torch.tensor([n], dtype=torch.int32).cuda(), return_lse=True)
    # every token counts n / 512 times over
    short = K.attention(q, kc, vc, torch.tensor([[0, 1]], dtype=torch.int32), torch.tensor([512], dtype=torch.int32), 0.125)
    tol = short[2] + (n / 16 / 2432 + 2432 + 64) * 2.0 ** -23      # longer chains, and the joining of all workers
    assert ((out.double().cpu() - short[0]).abs() <= tol).all()
    assert ((lse.double().cpu() - (short[1] + torch.log(torch.tensor(n / 512.0)))).abs() <= short[3] + 2.0 ** -12).all()


def test_large_expert_weights():
    """Weights of 2.3e9 elements each, of which those of the chosen experts hold numbers."""
    K_, F, E, top_k = 4096, 2200, 256, 2
    d = M.case(2, K_, 8, E, BF16, seed=3)
    chosen = [0, 3, E - 1, E - 2]
    d["Wr"].zero_()
    d["x"][:, :4] = torch.tensor([[3.0, 0, 0, 0], [0, 3.0, 0, 0]])
    for m in range(2):
        for s, e in enumerate((chosen[m], chosen[2 + m])):
            d["Wr"][e, m] = 4.0 - s
    g = K.generator(4)
    normal = lambda *s, std: (torch.randn(s, generator=g) * std).to(BF16)
    part = {"Wg": normal(4, F, K_, std=K_ ** -0.5), "Wu": normal(4, F, K_, std=K_ ** -0.5), "Wd": normal(4, K_, F, std=F ** -0.5)}
    full = {n: torch.empty((E, *t.shape[1:]), dtype=BF16, device="cuda") for n, t in part.items()}
    for n, t in part.items():
        for i, e in enumerate(chosen):
            full[n][e].copy_(t[i])
    got = ngr.fused_moe_swiglu(d["x"].cuda(), d["Wr"].cuda(), full["Wg"], full["Wu"], full["Wd"], top_k, norm=2, gamma=d["gamma"].cuda(),
                               return_routing=True)
    # the same layer of the four experts alone
    small = dict(d, Wr=d["Wr"][chosen], **part)
    want = M.reference(small, top_k)
    assert got[1].tolist() == [[chosen[0], chosen[2]], [chosen[1], chosen[3]]]
    # (the softmax runs over 256 experts there: the weights over the two chosen are the same)
    y = (got[0].cpu().double() - want[0]).abs()
    assert (y <= want[3]).all() and ((got[2].cpu() - want[2]).abs() <= want[4]).all()
