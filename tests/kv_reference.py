"""The rotated append and the paged attention in float64 on the CPU, and how
far a correct FP32 computation may be from them."""
import torch

U = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}      # half a step, relative
TINY = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}  # half a step among the subnormals


def generator(seed):
    g = torch.Generator("cpu")
    g.manual_seed(seed)
    return g


def pages_for(lengths, page_size, g, room=1, spare=2):
    """A block table for these lengths with pages in no order, -7 where a row needs none: (table, pages)."""
    have = [-(-max(n, 0) // page_size) for n in lengths]
    width = max(1, max(have) + room)
    total = sum(have) + spare
    order = torch.randperm(total, generator=g).to(torch.int32)
    table = torch.full((len(lengths), width), -7, dtype=torch.int32)
    at = 0
    for b, n in enumerate(have):
        table[b, :n] = order[at:at + n]
        at += n
    return table, total


def cache_like(pages, page_size, G, D, dtype, layout, g, fill=None):
    """A pair of caches [pages, page_size, G, D] in one of several layouts of memory."""
    shape = {"tokens": (pages, page_size, G, D), "heads": (pages, G, page_size, D), "joint": (pages, 2, page_size, G, D),
             "wide": (pages, page_size, G, D + 24), "pages inside": (page_size, pages, G, D)}[layout]

    def make():
        t = torch.randn(shape, generator=g) if fill is None else torch.full(shape, fill)
        return t.to(dtype)

    if layout == "joint":
        both = make()
        return both[:, 0], both[:, 1]
    view = {"tokens": lambda t: t, "heads": lambda t: t.transpose(1, 2), "wide": lambda t: t[..., 8:D + 8],
            "pages inside": lambda t: t.transpose(0, 1)}[layout]
    return view(make()), view(make())


def to_cuda(t):
    """The tensor on the GPU in the same layout of memory (views of one storage stay apart)."""
    out = torch.empty_strided(t.size(), t.stride(), dtype=t.dtype, device="cuda")
    return out.copy_(t)


# ------------------------------------------------------------------ append
def rotate(x, positions, inv_freq, interleaved):
    """x [T, heads, D] float64 rotated: (value, size of its terms)."""
    rot = 0 if inv_freq is None else 2 * inv_freq.numel()
    y, mag = x.clone(), x.abs()
    if rot == 0:
        return y, mag
    angle = positions.double()[:, None] * inv_freq.double()
    c, s = torch.cos(angle)[:, None], torch.sin(angle)[:, None]
    i = torch.arange(rot // 2)
    first, second = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
    a, b = x[..., first], x[..., second]
    y[..., first], y[..., second] = a * c - b * s, a * s + b * c
    mag[..., first] = mag[..., second] = a.abs() + b.abs()
    return y, mag


# cos and sin: 2 steps of 2^-24 each, the angle's own rounding to 24 bits of
# half a turn (pi 2^-25), two products and a sum of half a step 2^-24 each:
# below 2^-21 of |a| + |b|.
TURN = 2.0 ** -21


def check_rotated(got, val, mag, dtype, what):
    got = got.double().cpu()
    tol = U[dtype] * val.abs() + (1 + U[dtype]) * TURN * mag + TINY[dtype]
    over = (got - val).abs() - tol
    assert torch.isfinite(got).all(), what
    assert (over <= 0).all(), f"{what}: worst {((got - val).abs() / tol).max().item():.2f} times the tolerance"


# ------------------------------------------------------------------ attention
def attention(q, k_cache, v_cache, table, lengths, scale, window=0):
    """(out, lse, tolerance of out, of lse) for the rows in use; rows with a negative length are NaN."""
    dtype = q.dtype
    u, tiny = U[dtype], TINY[dtype]
    B, H, D = q.shape
    pages, size, G, _ = k_cache.shape
    out, lse, tol, tol_lse = (torch.full(s, float("nan"), dtype=torch.float64) for s in ((B, H, D), (B, H)) * 2)
    for b, n in enumerate(lengths.tolist()):
        if n < 0:
            continue
        n = min(n, table.shape[1] * size)
        j = torch.arange(max(0, n - window) if window else 0, n)
        page = table[b].long()[j // size]
        there = (page >= 0) & (page < pages)
        j, page = j[there], page[there]
        if len(j) == 0:
            out[b], lse[b], tol[b], tol_lse[b] = 0, -float("inf"), 0, 0
            continue
        k = k_cache[page, j % size].double().repeat_interleave(H // G, dim=1)     # [n, H, D]
        v = v_cache[page, j % size].double().repeat_interleave(H // G, dim=1)
        z = torch.einsum("hd,nhd->hn", q[b].double(), k) * scale
        size_z = torch.einsum("hd,nhd->hn", q[b].double().abs(), k.abs()) * abs(scale)
        lse[b] = torch.logsumexp(z, 1)
        p = torch.softmax(z, 1)
        out[b] = torch.einsum("hn,nhd->hd", p, v)
        # a score: D / 16 + 16 sums of up to a step 2^-23 of the terms'
        # sizes, then the scale, the difference to the maximum and exp2f, a
        # few steps of the score's own size and of 1
        dz = (D / 16 + 24) * 2.0 ** -23 * size_z + 2.0 ** -20
        # the weights: their scores' errors, and rounded once for the product
        # (independent roundings, taken at their worst); small ones are
        # subnormal; the sums' chain is a step for 16 tokens and 64 more for
        # the joining
        dp = p * (2 * dz.max(1, keepdim=True).values + u) + (tiny if dtype is torch.float16 else 0.0)
        chain = (len(j) / 16 + 64) * 2.0 ** -23
        tol[b] = torch.einsum("hn,nhd->hd", dp + chain * p, v.abs()) + u * out[b].abs() + tiny
        tol_lse[b] = dz.max(1).values + 2.0 ** -22 * (lse[b].abs() + z.abs().max(1).values) + chain
    return out, lse, tol, tol_lse


def check_attention(got, got_lse, want, what=""):
    out, lse, tol, tol_lse = want
    used = ~torch.isnan(lse)
    g = got.double().cpu()[used]
    assert torch.isfinite(g).all(), f"{what}: not finite"
    d = (g - out[used]).abs()
    assert (d <= tol[used]).all(), f"{what}: worst {(d / tol[used].clamp(min=1e-300)).max().item():.2f} times the tolerance"
    if got_lse is not None:
        gl, wl = got_lse.double().cpu()[used], lse[used]
        none = torch.isinf(wl)
        assert (gl[none] == wl[none]).all(), f"{what}: lse of empty rows"
        d = (gl[~none] - wl[~none]).abs()
        assert (d <= tol_lse[used][~none]).all(), f"{what}: lse {d.max().item():.3g}"
