"""Attention of one new token over a paged cache against its formula in
float64: lengths, pages, heads, layouts, windows, what is not to be looked at."""
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


def data(lengths, H, G, D, page_size, dtype, layout="tokens", seed=0, spread=2.0, dirty=True):
    g = R.generator(seed)
    B = len(lengths)
    table, pages = R.pages_for(lengths, page_size, g)
    k, v = R.cache_like(pages, page_size, G, D, dtype, layout, g)
    if dirty:      # slots that no sequence has hold anything
        held = torch.zeros((pages, page_size), dtype=torch.bool)
        for b, n in enumerate(lengths):
            j = torch.arange(max(n, 0))
            held[table[b].long()[j // page_size], j % page_size] = True
        k[~held] = float("nan")
        v[~held] = float("inf")
    q = (torch.randn((B, H, D), generator=g) * spread).to(dtype)
    return {"q": q, "k": k, "v": v, "table": table, "lengths": torch.tensor(lengths, dtype=torch.int32)}


def call(d, **kw):
    k, v = (R.to_cuda(d[n]) for n in "kv")
    return ngr.fused_paged_attention(R.to_cuda(d["q"]), k, v, d["table"].cuda(), d["lengths"].cuda(), return_lse=True, **kw)


def check(d, window=0, scale=None, what=""):
    D = d["q"].shape[-1]
    kw = {} if scale is None else {"scale": scale}
    out, lse = call(d, window=window, **kw)
    R.check_attention(out, lse, R.attention(d["q"], d["k"], d["v"], d["table"], d["lengths"], D ** -0.5 if scale is None else scale, window), what)
    return out, lse


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("D", [8, 64, 72, 80, 96, 128, 136, 192, 256])
def test_dimensions(D, dtype):
    check(data([37, 200, 1], 8, 2, D, 16, dtype, seed=D))


@pytest.mark.parametrize("H,G", [(1, 1), (8, 8), (8, 1), (16, 1), (17, 1), (40, 2), (64, 8), (71, 1), (12, 3), (128, 1)])
def test_heads(H, G):
    check(data([130, 5], H, G, 64, 16, BF16, seed=H))


@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 31, 32, 33, 47, 48, 63, 64, 65, 96, 97, 255, 256, 257, 1000])
def test_lengths(n):
    check(data([n], 8, 2, 128, 16, BF16, seed=n))


@pytest.mark.parametrize("page_size", [1, 2, 7, 16, 20, 33, 128, 1024])
@pytest.mark.parametrize("layout", ["tokens", "heads", "joint", "wide", "pages inside"])
def test_pages_and_layouts(page_size, layout):
    check(data([100, 3, 61], 6, 3, 64, page_size, F16, layout=layout, seed=page_size))


def test_ragged_batches():
    """Runs of tiles that begin and end inside sequences, many to a worker and many workers to one."""
    g = torch.Generator("cpu")
    g.manual_seed(8)
    check(data(torch.randint(0, 300, (150,), generator=g).tolist(), 8, 4, 64, 16, BF16))
    check(data([5000, 1, 0, 1, 700, 16, 3000], 8, 4, 128, 32, F16))
    check(data([9000], 4, 1, 64, 64, BF16))
    check(data([1] * 2000, 2, 2, 64, 1, F16))


@pytest.mark.parametrize("window", [1, 2, 15, 16, 17, 100, 10 ** 6, 1 << 40])
def test_windows(window):
    d = data([300, 16, 1, 17, 0, 95], 4, 2, 64, 16, BF16)
    # what lies before the window is not looked at: its pages may be anything
    for b, n in enumerate(d["lengths"].tolist()):
        d["table"][b, :max(0, n - min(window, 10 ** 6)) // 16] = 10 ** 6
    check(d, window=window)


def test_rows_without_tokens_and_rows_not_in_use():
    d = data([0, 40, -1, 0, -5, 7], 8, 2, 64, 16, F16)
    ref = R.attention(d["q"], d["k"], d["v"], d["table"], d["lengths"], 0.125)
    cuda = [R.to_cuda(d[k]) for k in ("q", "k", "v")] + [d["table"].cuda(), d["lengths"].cuda()]
    out = torch.full((6, 8, 64), 3.0, dtype=F16, device="cuda")
    lse = torch.full((6, 8), 4.0, device="cuda")
    got = ngr.fused_paged_attention(*cuda, out=out, lse=lse, return_lse=True)
    assert got[0] is out and got[1] is lse
    R.check_attention(out, lse, ref)
    for b in (2, 4):
        assert (out[b] == 3.0).all() and (lse[b] == 4.0).all()
    for b in (0, 3):
        assert (out[b] == 0).all() and (lse[b] == -float("inf")).all()
    # every row empty, or not in use
    none = torch.tensor([0, -1, 0, -1, 0, -1], dtype=torch.int32, device="cuda")
    out.fill_(3.0)
    ngr.fused_paged_attention(*cuda[:4], none, out=out)
    assert (out[0::2] == 0).all() and (out[1::2] == 3.0).all()


def test_scores_far_apart_and_equal():
    d = data([400, 90], 8, 2, 128, 16, BF16, spread=40.0)
    check(d)
    check(d, scale=-0.3)
    check(d, scale=1e-30)
    out, lse = check(d, scale=0.0)
    assert torch.allclose(lse.cpu(), torch.log(torch.tensor([[400.0], [90.0]])).expand(2, 8))


def test_infinite_scores():
    """Scores that are all -inf are as no tokens at all; +inf is NaN, as inf - inf is."""
    d = data([400, 90], 8, 2, 128, 16, BF16)
    d["k"].fill_(0)
    d["k"][..., 0] = 1
    d["q"][0, :, 0] = -float("inf")
    d["q"][1, :, 0] = float("inf")
    out, lse = call(d)
    assert (out[0] == 0).all() and (lse[0] == -float("inf")).all()
    assert torch.isnan(out[1]).all() and torch.isnan(lse[1]).all()


def test_infinite_and_nan_heads_stay_apart():
    """A query head that is not finite spoils its own row alone."""
    d = data([50, 600], 8, 2, 64, 16, F16)
    want = R.attention(d["q"], d["k"], d["v"], d["table"], d["lengths"], 0.125)
    d["q"][0, 1, 3] = float("nan")
    d["q"][1, 6, 0] = float("inf")
    out, lse = call(d)
    bad = torch.zeros((2, 8), dtype=torch.bool)
    bad[0, 1] = bad[1, 6] = True
    assert torch.isnan(out.cpu()[bad]).all()
    d = (out.cpu().double() - want[0])[~bad].abs()
    assert (d <= want[2][~bad]).all()


def test_strided_queries():
    d = data([70, 200, 9], 8, 4, 64, 16, BF16)
    wide = torch.randn((3, 16 * 64)).to(BF16)
    wide[:, 128:128 + 512] = d["q"].view(3, 512)
    d["q"] = wide[:, 128:128 + 512].view(3, 8, 64)
    check(d)
    d["q"] = d["q"].transpose(0, 1).contiguous().transpose(0, 1)
    check(d)


def test_tables_wider_and_of_more_rows():
    d = data([70, 200, 9], 8, 4, 64, 16, BF16)
    big = torch.full((5, 40), -1, dtype=torch.int32)
    big[:3, 2:2 + d["table"].shape[1]] = d["table"]
    want = R.attention(d["q"], d["k"], d["v"], d["table"], d["lengths"], 0.125)
    k, v = R.to_cuda(d["k"]), R.to_cuda(d["v"])
    out, lse = ngr.fused_paged_attention(d["q"].cuda(), k, v, big.cuda()[:, 2:30], d["lengths"].cuda(), return_lse=True)
    R.check_attention(out, lse, want)


def test_same_page_in_several_rows():
    """A prefix that sequences share."""
    d = data([64, 64, 90], 8, 2, 128, 16, F16, dirty=False)
    d["table"][1, :3] = d["table"][0, :3]
    d["table"][2, :2] = d["table"][0, 0]
    check(d)


@pytest.mark.parametrize("what", ["page too large", "page negative", "length past the table"])
def test_bad_pages_are_left_out_and_reported(what):
    d = data([100, 40, 70], 8, 2, 64, 16, BF16, dirty=False)
    if what == "page too large":
        d["table"][1, 1] = d["k"].shape[0]
    elif what == "page negative":
        d["table"][1, 1] = -1
    else:
        d["lengths"][0] = d["table"].shape[1] * 16 + 5
        d["table"][0] = 0
    want = R.attention(d["q"], d["k"], d["v"], d["table"], d["lengths"], 0.125)
    n = ngr.binding.ngr_paged_attention_workspace_bytes(3, 8, 2, 64, d["table"].shape[1] * 16, 0)
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
    out, lse = call(d, workspace=ws)
    R.check_attention(out, lse, want, what)
    with pytest.raises(ngr.NgrError) as e:
        ngr.check_workspace(ws)
    assert e.value.status == -9
    good = data([100, 40, 70], 8, 2, 64, 16, BF16)
    call(good, workspace=ws)
    ngr.check_workspace(ws)


def test_same_bits_twice():
    d = data([5000, 33, 800], 16, 2, 128, 16, BF16)
    a, b = call(d), call(d)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_joined_by_lse():
    """Results over two parts of a context, joined by their lse, are the result over all of it."""
    d = data([320], 8, 2, 64, 16, F16)
    want = R.attention(d["q"], d["k"], d["v"], d["table"], d["lengths"], 0.125)
    parts = []
    for at, n in ((0, 160), (10, 160)):
        e = dict(d, table=d["table"][:, at:].contiguous(), lengths=torch.tensor([n], dtype=torch.int32))
        parts.append([t.double().cpu() for t in call(e)])
    total = torch.logaddexp(parts[0][1], parts[1][1])
    out = sum(o * torch.exp(l - total)[..., None] for o, l in parts)
    # (each part is rounded once more: half a step of its size)
    extra = R.U[F16] * sum((o * torch.exp(l - total)[..., None]).abs() for o, l in parts)
    assert ((out - want[0]).abs() <= 2 * want[2] + extra).all()
    assert ((total - want[1]).abs() <= 2 * want[3] + 1e-6).all()


@pytest.mark.parametrize("page_size", [1, 16])
@pytest.mark.parametrize("B", [1, 140, 200])
def test_bad_pages_of_many_rows_are_reported(B, page_size):
    """Any row's last page, or its length: found in batches of every size, and only then."""
    lengths = [40 + b % 300 for b in range(B)]
    for row in sorted({0, B // 2, B - 1}):
        for what in ("none", "page", "length"):
            d = data(lengths, 4, 1, 64, page_size, BF16, dirty=False, seed=row)
            if what == "page":
                d["table"][row, (lengths[row] - 1) // page_size] = d["k"].shape[0]
            elif what == "length":
                d["table"][row] = 0
                d["lengths"][row] = d["table"].shape[1] * page_size + 1
            n = ngr.binding.ngr_paged_attention_workspace_bytes(B, 4, 1, 64, d["table"].shape[1] * page_size, 0)
            ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
            out, lse = call(d, workspace=ws)
            R.check_attention(out, lse, R.attention(d["q"], d["k"], d["v"], d["table"], d["lengths"], 0.125), what)
            if what == "none":
                ngr.check_workspace(ws)
            else:
                with pytest.raises(ngr.NgrError) as e:
                    ngr.check_workspace(ws)
                assert e.value.status == -9


@pytest.mark.parametrize("lengths,H,G,D", [([2500] * 18, 16, 8, 64), ([2000] * 3 + [1, 0, 1700] * 5, 8, 8, 128), ([700] * 151, 2, 1, 256),
                                           ([700] * 152, 2, 1, 256), ([900, 3, 16] * 8, 40, 2, 256)])
def test_batches_that_nearly_fill_the_device(lengths, H, G, D):
    check(data(lengths, H, G, D, 32, F16, seed=len(lengths)))


def test_values_in_another_layout_than_keys():
    """The strides of k and v are their own."""
    for lengths in ([100, 3, 61], [700] * 60):
        d = data(lengths, 8, 4, 64, 16, BF16, layout="tokens")
        for layout in ("heads", "wide", "pages inside"):
            other = R.cache_like(d["k"].shape[0], 16, 4, 64, BF16, layout, R.generator(1), fill=0.0)[1]
            d["v"] = other.copy_(d["v"])
            check(d, what=layout)


def test_output_in_the_queries_place():
    for lengths in ([100, 0, -1, 61], [5000, 40] + [300] * 100):
        d = data(lengths, 16, 4, 64, 16, F16)
        want, want_lse = call(d, out=torch.zeros_like(d["q"], device="cuda"))
        q = d["q"].cuda()
        out, lse = ngr.fused_paged_attention(q, R.to_cuda(d["k"]), R.to_cuda(d["v"]), d["table"].cuda(), d["lengths"].cuda(), out=q,
                                             return_lse=True)
        used = d["lengths"] >= 0
        assert out is q and torch.equal(q.cpu()[used], want.cpu()[used]) and torch.equal(lse.cpu()[used], want_lse.cpu()[used])
        assert torch.equal(q.cpu()[~used], d["q"][~used])


@pytest.mark.parametrize("G,group,D", [(700, 9, 136), (1300, 1, 192), (608, 9, 256), (2500, 1, 16)])
def test_more_heads_than_the_device_has_warps(G, group, D):
    d = data([70, 3, 0], G * group, G, D, 16, F16, seed=G, dirty=False)
    check(d)
    d["table"][1, 0] = d["k"].shape[0]
    n = ngr.binding.ngr_paged_attention_workspace_bytes(3, G * group, G, D, d["table"].shape[1] * 16, 0)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    call(d, workspace=ws)
    with pytest.raises(ngr.NgrError):
        ngr.check_workspace(ws)
