"""The rotated append to a paged cache against its formula in float64: every
element written, every other one untouched."""
import pytest
import torch

import normalization_gemm_row_gb300 as ngr
import kv_reference as R

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _built():
    ngr.build()
    torch.cuda.init()


def frequencies(rot, theta=10000.0):
    return (theta ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)).float() if rot else None


def run(T, H, G, D, page_size, dtype, rot=None, interleaved=False, layout="tokens", positions=None, rows=None, sequences=None,
        seed=0, apart=False, in_place=False, offset=0):
    """One call with slices of one QKV array (or tensors of their own), checked whole."""
    g = R.generator(seed)
    rot = D if rot is None else rot
    positions = torch.tensor(positions if positions is not None else [3 * t for t in range(T)], dtype=torch.int32)
    rows_cpu = torch.tensor(rows, dtype=torch.int32) if rows is not None else None
    B = sequences or T
    row_of = rows_cpu if rows_cpu is not None else torch.arange(T, dtype=torch.int32)
    lengths = [0] * B
    for r, p in zip(row_of.tolist(), positions.tolist()):
        if p >= 0:
            lengths[r] = max(lengths[r], p + 1)
    table, pages = R.pages_for(lengths, page_size, g)
    k_cache, v_cache = R.cache_like(pages, page_size, G, D, dtype, layout, g)
    inv = frequencies(rot)
    wide = torch.randn((T, (H + 2 * G) * D + offset), generator=g).to(dtype)
    qkv = wide[:, offset:]
    cuda = wide.cuda()[:, offset:]
    parts = [(t[:, :H * D].view(T, H, D), t[:, H * D:(H + G) * D].view(T, G, D), t[:, (H + G) * D:].view(T, G, D)) for t in (qkv, cuda)]
    (q, k, v), (cq, ck, cv) = parts
    if apart:
        cq, ck, cv = cq.contiguous(), ck.transpose(0, 1).contiguous().transpose(0, 1), cv.contiguous()
    if layout == "joint":
        both = torch.stack((k_cache, v_cache), 1).cuda()
        kc, vc = both[:, 0], both[:, 1]
    else:
        kc, vc = R.to_cuda(k_cache), R.to_cuda(v_cache)
    ws = torch.full((256,), 255, dtype=torch.uint8, device="cuda")
    q_in = cq.clone()
    out = cq if in_place else torch.full((T, H, D), 7.0, dtype=dtype, device="cuda")
    got = ngr.fused_rope_append_kv(cq, ck, cv, kc, vc, table.cuda(), positions.cuda(), rows=rows_cpu.cuda() if rows_cpu is not None else None,
                                   inv_freq=inv.cuda() if inv is not None else None, interleaved=interleaved, q_out=out, workspace=ws)
    assert got is out
    ngr.check_workspace(ws)
    used = positions >= 0
    val, mag = R.rotate(q.double(), positions, inv, interleaved)
    R.check_rotated(got.cpu()[used], val[used], mag[used], dtype, "q")
    left = q_in.cpu() if in_place else torch.full((T, H, D), 7.0, dtype=dtype)
    assert torch.equal(got.cpu()[~used], left[~used])
    val, mag = R.rotate(k.double(), positions, inv, interleaved)
    page = table[row_of.long()[used], (positions[used] // page_size).long()].long()
    slot = (positions[used] % page_size).long()
    new_k, new_v = kc.cpu(), vc.cpu()
    R.check_rotated(new_k[page, slot], val[used], mag[used], dtype, "k")
    assert torch.equal(new_v[page, slot], v[used])
    # nothing else is touched
    for new, old in ((new_k, k_cache), (new_v, v_cache)):
        new, old = new.clone(), old.clone()
        new[page, slot] = 0
        old[page, slot] = 0
        assert torch.equal(new, old)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,rot", [(128, 128), (64, 64), (80, 32), (80, 40), (80, 20), (256, 64), (96, 0), (72, 72), (5, 4), (2, 2)])
def test_dimensions(D, rot, interleaved, dtype):
    run(5, 4, 2, D, 16, dtype, rot=rot, interleaved=interleaved)


@pytest.mark.parametrize("layout", ["tokens", "heads", "joint", "wide", "pages inside"])
@pytest.mark.parametrize("page_size", [1, 3, 16, 20, 256])
def test_pages_and_layouts(page_size, layout):
    run(9, 6, 3, 64, page_size, BF16, layout=layout, positions=[0, 1, page_size - 1, page_size, 2 * page_size + 1, 40, 77, 5, 300])


@pytest.mark.parametrize("T,H,G", [(1, 64, 8), (1, 1, 1), (3, 7, 7), (300, 2, 1), (33, 71, 1), (2, 128, 16)])
def test_heads_and_tokens(T, H, G):
    run(T, H, G, 128, 32, F16, positions=[(7 * t) % 90 for t in range(T)])


@pytest.mark.parametrize("offset", [1, 2, 4])
@pytest.mark.parametrize("interleaved", [False, True])
def test_addresses_off_the_boundary(offset, interleaved):
    run(4, 3, 2, 32, 8, BF16, interleaved=interleaved, offset=offset, layout="wide")


def test_prompts_of_several_sequences():
    runs = [3, 0, 41, 1]
    rows = [b for b, n in enumerate(runs) for _ in range(n)]
    run(45, 8, 4, 64, 16, F16, positions=[5 + j for n in runs for j in range(n)], rows=rows, sequences=4)


def test_tokens_left_out_and_in_place():
    for in_place in (False, True):
        run(6, 4, 2, 64, 16, BF16, positions=[0, -1, 17, -5, 3, 31], in_place=in_place)
    run(3, 4, 2, 64, 16, BF16, positions=[-1, -1, -1])


def test_tensors_apart():
    run(6, 4, 2, 64, 16, BF16, apart=True)


@pytest.mark.parametrize("position", [1, 1000, 131071, 1 << 20, (1 << 31) - 1])
def test_far_positions(position):
    """Angles of far positions: one page at the end of a long table."""
    D, size = 128, 1 << 20
    g = R.generator(3)
    q, k, v = (torch.randn((1, 2, D), generator=g).to(F16) for _ in range(3))
    width = position // size + 1
    table = torch.full((1, width), -1, dtype=torch.int32)
    table[0, -1] = 0
    inv = frequencies(D, 500000.0)
    # (slots of one page that overlap in memory would be refused; the page is real)
    kc = torch.zeros((1, size, 2, D), dtype=F16, device="cuda")
    vc = torch.zeros_like(kc)
    positions = torch.tensor([position], dtype=torch.int32)
    got = ngr.fused_rope_append_kv(q.cuda(), k.cuda(), v.cuda(), kc, vc, table.cuda(), positions.cuda(), inv_freq=inv.cuda())
    val, mag = R.rotate(q.double(), positions, inv, False)
    R.check_rotated(got, val, mag, F16, "q")
    val, mag = R.rotate(k.double(), positions, inv, False)
    R.check_rotated(kc[0, position % size].cpu()[None], val, mag, F16, "k")
    assert torch.equal(vc[0, position % size].cpu()[None], v)


def test_frequencies_of_all_sizes():
    """Any finite float: negative, above one, subnormal, zero."""
    inv = torch.tensor([1.0, -1.0, 3.0e4, -2.5, 1e-30, 1e-42, 0.0, 6.2831855, 1.0e-7, 16777216.0, 0.5, 0.3, 3.1415927, -0.0, 100.5, 2.0 ** -60])
    D = 32
    g = R.generator(4)
    q = torch.randn((3, 1, D), generator=g).to(BF16)
    k, v = q.clone(), q.clone()
    positions = torch.tensor([7, 12345, 99999], dtype=torch.int32)
    table = torch.arange(3, dtype=torch.int32)[:, None].repeat(1, 2000)
    kc = torch.zeros((3, 64, 1, D), dtype=BF16, device="cuda")
    vc = torch.zeros_like(kc)
    got = ngr.fused_rope_append_kv(q.cuda(), k.cuda(), v.cuda(), kc, vc, table.cuda(), positions.cuda(), inv_freq=inv.cuda())
    # exact angles in rationals: position x float is exact in integers, the turn by mpmath-free high precision
    from fractions import Fraction
    two_pi = 2 * Fraction(31415926535897932384626433832795028841971693993751058209749445923, 10 ** 64)
    angle = torch.zeros((3, D // 2), dtype=torch.float64)
    for t, p in enumerate(positions.tolist()):
        for i, f in enumerate(inv.tolist()):
            x = Fraction(f) * p
            angle[t, i] = float(x - two_pi * (x / two_pi).__floor__())
    c, s = torch.cos(angle)[:, None], torch.sin(angle)[:, None]
    a, b = q.double()[..., :D // 2], q.double()[..., D // 2:]
    val = torch.cat((a * c - b * s, a * s + b * c), -1)
    mag = torch.cat((a.abs() + b.abs(),) * 2, -1)
    R.check_rotated(got, val, mag, BF16, "q")


def test_without_queries():
    g = R.generator(5)
    k, v = torch.randn((2, 3, 64), generator=g).to(F16), torch.randn((2, 3, 64), generator=g).to(F16)
    kc, vc = torch.zeros((2, 4, 3, 64), dtype=F16, device="cuda"), torch.zeros((2, 4, 3, 64), dtype=F16, device="cuda")
    table = torch.tensor([[1], [0]], dtype=torch.int32, device="cuda")
    pos = torch.tensor([2, 3], dtype=torch.int32, device="cuda")
    assert ngr.fused_rope_append_kv(None, k.cuda(), v.cuda(), kc, vc, table, pos) is None
    assert torch.equal(kc[1, 2].cpu(), k[0]) and torch.equal(kc[0, 3].cpu(), k[1]) and torch.equal(vc[1, 2].cpu(), v[0])


@pytest.mark.parametrize("what", ["page too large", "page negative", "position past the table", "row past the table", "row negative"])
def test_bad_tokens_are_left_out_and_reported(what):
    g = R.generator(6)
    T, G, D, size = 4, 2, 64, 8
    q, k, v = (torch.randn((T, G, D), generator=g).to(F16).cuda() for _ in range(3))
    table = torch.tensor([[0, 1], [2, 3], [4, 5], [6, 7]], dtype=torch.int32)
    positions = torch.tensor([3, 9, 0, 15], dtype=torch.int32)
    rows = torch.arange(4, dtype=torch.int32)
    if what == "page too large":
        table[1, 1] = 8
    elif what == "page negative":
        table[1, 1] = -1
    elif what == "position past the table":
        positions[1] = 16
    elif what == "row past the table":
        rows[1] = 4
    else:
        rows[1] = -1
    kc = torch.zeros((8, size, G, D), dtype=F16, device="cuda")
    vc = torch.zeros_like(kc)
    out = torch.full_like(q, 9.0)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    ngr.fused_rope_append_kv(q, k, v, kc, vc, table.cuda(), positions.cuda(), rows=rows.cuda(), q_out=out, workspace=ws)
    with pytest.raises(ngr.NgrError) as e:
        ngr.check_workspace(ws)
    assert e.value.status == -9
    assert (out[1] == 9.0).all() and torch.equal(out[0], q[0]) and torch.equal(out[3], q[3])
    want = torch.zeros_like(vc)
    for t in (0, 2, 3):
        want[table[t, positions[t] // size].item(), positions[t].item() % size] = v[t]
    assert torch.equal(vc, want)
    # the next call clears the report, and a call without a workspace leaves the token out too
    good = torch.tensor([3, 1, 0, 15], dtype=torch.int32, device="cuda")
    ws.fill_(255)
    ngr.fused_rope_append_kv(q, k, v, kc, vc, torch.arange(8, dtype=torch.int32, device="cuda").view(4, 2), good, workspace=ws)
    ngr.check_workspace(ws)
    before = vc.clone()
    ngr.fused_rope_append_kv(q, k, v, kc, vc, table.cuda(), positions.cuda(), rows=rows.cuda())
    assert torch.equal(vc[table[0, 0].item(), 3], v[0])
    assert torch.equal(vc[3], before[3]) or what == "row past the table"


@pytest.mark.parametrize("layout", ["heads", "wide", "pages inside"])
def test_values_in_another_layout_than_keys(layout):
    """The strides of the two caches are their own."""
    g = R.generator(6)
    k, v = torch.randn((4, 3, 64), generator=g).to(BF16), torch.randn((4, 3, 64), generator=g).to(BF16)
    kc = torch.zeros((5, 16, 3, 64), dtype=BF16, device="cuda")
    vc = R.to_cuda(R.cache_like(5, 16, 3, 64, BF16, layout, g, fill=0.0)[1])
    table = torch.tensor([[4, 1], [0, 3]], dtype=torch.int32)
    rows, pos = torch.tensor([0, 0, 1, 1], dtype=torch.int32), torch.tensor([15, 16, 3, 31], dtype=torch.int32)
    ngr.fused_rope_append_kv(None, k.cuda(), v.cuda(), kc, vc, table.cuda(), pos.cuda(), rows=rows.cuda())
    page, slot = table[rows.long(), pos.long() // 16].long(), pos.long() % 16
    for got, new in ((kc.cpu(), k), (vc.cpu(), v)):
        assert torch.equal(got[page, slot], new)
        got = got.clone()
        got[page, slot] = 0
        assert (got == 0).all()
