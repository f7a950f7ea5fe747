"""What is measured of the operators of a decode step between a block's products.

Three operators:

- ``append``: new tokens' keys and values into a paged cache, keys and queries rotated by their
  position on the way:
      angle = position * inv_freq[i],  (a, b) -> (a cos - b sin, a sin + b cos),
      cache[table[row, position // page], position % page] = key, value
- ``attend``: attention of one new token for each sequence over the paged cache:
      s_j = scale q . k_j,  lse = log sum_j exp s_j,  out = sum_j exp(s_j - lse) v_j,
  j over the sequence's tokens, or the last ``window`` of them; no tokens: out = 0, lse = -inf
- ``moe``: a whole mixture-of-experts layer for a few tokens:
      a = RMSNorm(x),  p = softmax(a Wr^T),  the top_k largest p (ties: the lowest expert) over their sum,
      y = sum_e p_e (SiLU(a Wg_e^T) * (a Wu_e^T)) Wd_e^T

``run`` computes them in plain torch operations in 32 bits (angles in 64), or (``own``) calls the
framework's entry points.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
EPS = 1e-5
THETA = 500000.0


# ---------------------------------------------------------------- cases
def _append(name, T, B, past, H, G, D, page, dtype, rot=None, interleaved=False):
    """T new tokens, T // B or one more for each of B sequences that have ``past`` tokens each."""
    return {"name": name, "op": "append", "T": T, "B": B, "past": past, "H": H, "G": G, "D": D, "page": page,
            "dtype": dtype, "rot": D if rot is None else rot, "interleaved": interleaved}


def _attend(name, B, length, H, G, D, page, dtype, ragged=0.0, empty=0, window=0, head_major=False):
    """B sequences of ``length`` tokens down to (1 - ragged) of it, ``empty`` of them without any."""
    return {"name": name, "op": "attend", "B": B, "length": length, "H": H, "G": G, "D": D, "page": page,
            "dtype": dtype, "ragged": ragged, "empty": empty, "window": window, "head_major": head_major}


def _moe(name, M, K, F, E, k, dtype):
    return {"name": name, "op": "moe", "M": M, "K": K, "F": F, "E": E, "k": k, "dtype": dtype}


def listed():
    return [
        # one sequence's new token in a block of width 8192: latency
        _append("append_token", 1, 1, 1000, 64, 8, 128, 16, "bf16"),
        # a decode step of a full batch, far into its contexts
        _append("append_batch", 256, 256, 100000, 32, 8, 128, 32, "bf16"),
        # prompts on their way into the cache
        _append("append_prompt", 8192, 4, 0, 64, 8, 128, 64, "f16"),
        # a ragged chunk of prompts, heads of 80 with 32 rotated dimensions in neighbouring pairs
        _append("append_ragged", 1021, 7, 333, 10, 5, 80, 20, "f16", rot=32, interleaved=True),
        # one sequence, a short context: latency
        _attend("attend_token", 1, 1000, 64, 8, 128, 16, "bf16"),
        # one sequence, a long context: the work is split over its length
        _attend("attend_long", 1, 131072, 64, 8, 128, 64, "bf16"),
        # a serving batch at lengths between a quarter and all of 8192
        _attend("attend_batch", 64, 8192, 64, 8, 128, 16, "bf16", ragged=0.75),
        # as many key heads as query heads, heads of 80, some rows unused, a window, pages by heads
        _attend("attend_ragged", 37, 5003, 12, 12, 80, 20, "f16", ragged=0.98, empty=3, window=2048, head_major=True),
        # one token through a few wide experts: the chosen ones' weights are read once
        _moe("moe_token", 1, 4096, 14336, 8, 2, "bf16"),
        # a small batch through many narrow experts
        _moe("moe_fine", 8, 2048, 768, 128, 8, "bf16"),
        # a full decode batch: nearly every expert is chosen by somebody
        _moe("moe_batch", 32, 4096, 1536, 64, 6, "bf16"),
        # odd sizes
        _moe("moe_ragged", 5, 1000, 2001, 13, 3, "f16"),
    ]


def _spread(rng, low, high):
    """A whole number whose logarithm is spread evenly over [low, high]."""
    return min(high, max(low, round(math.exp(rng.uniform(math.log(low), math.log(high + 1))))))


def draw(rng):
    dtype = rng.choice(["bf16", "f16"])
    op = rng.choice(["append", "attend", "attend", "moe"])
    if op == "moe":
        while True:
            M, K, F, E = _spread(rng, 1, 32), _spread(rng, 64, 8192), _spread(rng, 64, 14336), _spread(rng, 2, 160)
            if rng.random() < 0.75:
                K, F = -(-K // 64) * 64, -(-F // 64) * 64
            k = rng.randint(1, min(8, E))
            if E * F * K <= 1 << 29 and M * k * F * K <= 1 << 31:
                break
        c = _moe("", M, K, F, E, k, dtype)
    else:
        G = rng.choice([1, 2, 3, 4, 8, 8, 16])
        H = G * rng.choice([1, 1, 2, 4, 7, 8, 8, 16])
        D = rng.choice([64, 64, 80, 96, 128, 128, 128, 192, 256])
        page = rng.choice([1, 8, 16, 16, 20, 32, 64, 64, 128, 256])
        if op == "append":
            T = _spread(rng, 1, 8192)
            while T * (H + 2 * G) * D > 1 << 26:
                T = T // 2 + 1
            B = T if rng.random() < 0.4 else rng.randint(1, min(T, 16))
            c = _append("", T, B, _spread(rng, 1, 8192) - 1 if B < 64 else rng.randint(0, 300), H, G, D, page, dtype,
                        rot=D // rng.choice([1, 1, 2, 4]), interleaved=rng.random() < 0.4)
        else:
            B, length = _spread(rng, 1, 256), _spread(rng, 1, 131072)
            while B * length * max(G * D, 512) > 1 << 28:
                B, length = B // 2 + 1, length // 2 + 1
            c = _attend("", B, length, H, G, D, page, dtype, ragged=rng.choice([0.0, rng.random(), 0.9]),
                        empty=rng.choice([0, 0, rng.randint(0, B - 1)]),
                        window=rng.choice([0, 0, _spread(rng, 1, 8192)]), head_major=rng.random() < 0.3)
    del c["name"]
    return c


def _lengths(case):
    """The sequences' lengths, longest first."""
    B, L = case["B"], case["length"]
    live = B - case["empty"]
    return [max(1, round(L * (1.0 - case["ragged"] * i / max(1, live - 1)))) for i in range(live)] + [0] * case["empty"]


def _runs(case):
    """New tokens of each sequence."""
    T, B = case["T"], case["B"]
    return [T // B + (i < T % B) for i in range(B)]


# --------------------------------------------------------------- inputs
def _pages(first, last, page, room, g):
    """A block table for sequences whose tokens [first, last) are in the cache, with ``room`` tokens to grow, its pages
    in no order; -1 where a sequence has none.  (table, pages in all)"""
    at = torch.arange(-(-(max(last) + room) // page))
    low = torch.tensor(first)[:, None] // page
    high = -(-torch.tensor(last)[:, None] // page)
    held = ((at >= low) & (at < high)).cuda()
    total = int(held.sum()) + 3
    table = torch.full(held.shape, -1, dtype=torch.int32, device="cuda")
    table[held] = torch.randperm(total, generator=g, device="cuda")[:total - 3].to(torch.int32)
    return table, total


def prepare(case, seed):
    g = torch.Generator("cuda")
    g.manual_seed(seed)
    rng = random.Random(seed)
    dt = DTYPES[case["dtype"]]

    def normal(*shape, std=1.0, mean=0.0):
        """Drawn in pieces, rounded at once."""
        out = torch.empty(shape, dtype=dt, device="cuda")
        flat = out.view(-1)
        for at in range(0, flat.numel(), 1 << 28):
            part = flat[at:at + (1 << 28)]
            part.copy_(torch.randn(part.numel(), generator=g, device="cuda").mul_(std).add_(mean))
        return out

    s = {"case": case}
    if case["op"] == "moe":
        M, K, F, E, k = (case[n] for n in ("M", "K", "F", "E", "k"))
        s["gamma"] = normal(K, std=0.1, mean=1.0)
        s["Wr"] = normal(E, K, std=1.5 * K ** -0.5)
        s["Wg"], s["Wu"] = normal(E, F, K, std=K ** -0.5), normal(E, F, K, std=K ** -0.5)
        s["Wd"] = normal(E, K, F, std=F ** -0.5)
        # of more tokens than needed, those come first whose choice of experts does not hang on a rounding
        x = normal(2 * M + 16, K, mean=0.1)
        a = x.double() * torch.rsqrt((x.double() ** 2).mean(-1, keepdim=True) + EPS) * s["gamma"].double()
        z = torch.sort(a @ s["Wr"].double().t(), dim=-1, descending=True).values[:, :k + 1]
        gap = (z[:, :-1] - z[:, 1:]).min(-1).values if z.shape[1] > 1 else z[:, 0].abs() + 1
        s["x"] = x[torch.argsort((gap < 1e-3).to(torch.int8), stable=True)[:M]].contiguous()
        return s
    H, G, D, page, B = (case[n] for n in ("H", "G", "D", "page", "B"))
    if case["op"] == "append":
        T, rot, past = case["T"], case["rot"], case["past"]
        runs = _runs(case)
        # (what the sequences have from before lies in other pages, which the call does not touch)
        s["table"], pages = _pages([past] * B, [past + n for n in runs], page, 64, g)
        # the products' output: queries, keys and values of a token side by side
        s["qkv"] = normal(T, (H + 2 * G) * D)
        s["q"] = s["qkv"][:, :H * D].view(T, H, D)
        s["k"] = s["qkv"][:, H * D:(H + G) * D].view(T, G, D)
        s["v"] = s["qkv"][:, (H + G) * D:].view(T, G, D)
        s["positions"] = torch.tensor([past + j for n in runs for j in range(n)], dtype=torch.int32, device="cuda")
        s["rows"] = torch.tensor([b for b, n in enumerate(runs) for _ in range(n)], dtype=torch.int32, device="cuda")
        s["inv_freq"] = (THETA ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)).float().cuda()
    else:
        lengths = _lengths(case)
        rng.shuffle(lengths)
        s["table"], pages = _pages([0] * B, lengths, page, case["length"] // 4 + 1, g)
        s["lengths"] = torch.tensor(lengths, dtype=torch.int32, device="cuda")
        s["q"] = normal(B, H, D, std=2.0)     # scores that make some tokens count far more than others
    if case.get("head_major"):
        s["k_cache"], s["v_cache"] = (normal(pages, G, page, D).transpose(1, 2) for _ in range(2))
    else:
        s["k_cache"], s["v_cache"] = normal(pages, page, G, D), normal(pages, page, G, D)
    return s


# ------------------------------------------------------------ plain forms
def _rotated(x, cos, sin, rot, interleaved):
    """x [T, heads, D] with its first ``rot`` dimensions rotated; cos, sin [T, rot / 2]."""
    y = x.float()
    turn, rest = y[..., :rot], y[..., rot:]
    cos, sin = cos[:, None], sin[:, None]
    if interleaved:
        a, b = turn[..., 0::2], turn[..., 1::2]
        turn = torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)
    else:
        a, b = turn[..., :rot // 2], turn[..., rot // 2:]
        turn = torch.cat((a * cos - b * sin, a * sin + b * cos), -1)
    return torch.cat((turn, rest), -1).to(x.dtype)


def _append_plain(s):
    c = s["case"]
    angle = s["positions"].double()[:, None] * s["inv_freq"].double()
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    position = s["positions"].long()
    page = s["table"][s["rows"].long(), position // c["page"]].long()
    slot = position % c["page"]
    s["k_cache"][page, slot] = _rotated(s["k"], cos, sin, c["rot"], c["interleaved"])
    s["v_cache"][page, slot] = s["v"]
    return {"q": _rotated(s["q"], cos, sin, c["rot"], c["interleaved"]), "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _attend_plain(s):
    c = s["case"]
    B, H, G, D, L = c["B"], c["H"], c["G"], c["D"], c["length"]
    table = s["table"][:, :-(-L // c["page"])].clamp(min=0).long()
    at = torch.arange(L, device="cuda")
    n = s["lengths"][:, None]
    seen = at < n
    if c["window"]:
        seen = seen & (at >= n - c["window"])
    k = s["k_cache"][table].flatten(1, 2)[:, :L].float()
    z = torch.matmul(s["q"].view(B, G, H // G, D).float(), k.permute(0, 2, 3, 1)) * D ** -0.5
    del k
    z = torch.where(seen[:, None, None], z, -math.inf)
    top = z.max(-1, keepdim=True).values
    top = torch.where(top > -math.inf, top, 0.0)
    p = torch.exp(z - top)
    del z
    total = p.sum(-1, keepdim=True)
    v = torch.where(seen[:, :, None, None], s["v_cache"][table].flatten(1, 2)[:, :L].float(), 0.0)
    out = torch.matmul(p, v.transpose(1, 2)) / torch.where(total > 0, total, 1.0)
    return {"out": out.reshape(B, H, D).to(s["q"].dtype), "lse": (torch.log(total) + top).reshape(B, H)}


def _moe_plain(s):
    c = s["case"]
    k = c["k"]
    x = s["x"].float()
    a = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * s["gamma"].float()
    z = a @ s["Wr"].float().t()
    p = torch.exp(z - z.max(-1, keepdim=True).values)
    p = p / p.sum(-1, keepdim=True)
    experts = torch.sort(p, dim=-1, descending=True, stable=True).indices[:, :k]
    w = p.gather(1, experts)
    w = w / w.sum(-1, keepdim=True)
    col = a[:, None, :, None]
    gate = torch.matmul(s["Wg"][experts].float(), col)
    up = torch.matmul(s["Wu"][experts].float(), col)
    h = gate / (1.0 + torch.exp(-gate)) * up * w[:, :, None, None]
    y = torch.matmul(s["Wd"][experts].float(), h).sum(1)[..., 0]
    return {"y": y.to(s["x"].dtype), "experts": experts.to(torch.int32), "weights": w}


# ------------------------------------------------------- the framework's calls
def _append_own(s):
    import normalization_gemm_row_gb300 as ngr
    q = ngr.fused_rope_append_kv(s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"], s["table"], s["positions"],
                                 rows=s["rows"], inv_freq=s["inv_freq"], interleaved=s["case"]["interleaved"])
    return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _attend_own(s):
    import normalization_gemm_row_gb300 as ngr
    out, lse = ngr.fused_paged_attention(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lengths"],
                                         window=s["case"]["window"], return_lse=True)
    return {"out": out, "lse": lse}


def _moe_own(s):
    import normalization_gemm_row_gb300 as ngr
    y, experts, weights = ngr.fused_moe_swiglu(s["x"], s["Wr"], s["Wg"], s["Wu"], s["Wd"], s["case"]["k"], norm=ngr.NORM_RMS,
                                               gamma=s["gamma"], eps=EPS, renormalize=True, return_routing=True)
    return {"y": y, "experts": experts, "weights": weights}


def run(state):
    op = state["case"]["op"]
    if op == "append":
        return _append_own(state) if own else _append_plain(state)
    if op == "attend":
        return _attend_own(state) if own else _attend_plain(state)
    return _moe_own(state) if own else _moe_plain(state)


# ----------------------------------------------------------- work and truth
def work(case):
    if case["op"] == "moe":
        M, K, F, E, k = (case[n] for n in ("M", "K", "F", "E", "k"))
        # (the experts that somebody chooses: their mean number for even choices)
        chosen = E * (1.0 - (1.0 - k / E) ** M)
        return {"bytes": int(6 * chosen * F * K) + 2 * (E + 1) * K + 4 * M * K + 8 * M * k,
                "flops": 6 * M * k * F * K + 2 * M * E * K}
    H, G, D = case["H"], case["G"], case["D"]
    if case["op"] == "append":
        T = case["T"]
        return {"bytes": 4 * T * (H + 2 * G) * D + 12 * T, "flops": 3 * T * (H + G) * case["rot"]}
    seen = sum(min(n, case["window"]) if case["window"] else n for n in _lengths(case))
    return {"bytes": 4 * seen * G * D + 4 * case["B"] * H * (D + 1), "flops": 4 * seen * H * D}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "append":
        rot, half = case["rot"], case["rot"] // 2
        pos = s["positions"].long()
        phase = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), torch.outer(pos.double(), s["inv_freq"].double()))
        first = torch.arange(half, device="cuda") * (2 if case["interleaved"] else 1)
        second = first + (1 if case["interleaved"] else half)

        def turn(x):
            y = x.double()
            z = torch.complex(y[..., first], y[..., second]) * phase[:, None]
            y[..., first], y[..., second] = z.real, z.imag
            return y

        where = s["table"].long()[s["rows"].long(), pos // case["page"]], pos % case["page"]
        out = {"q": turn(s["q"]), "k_cache": s["k_cache"].double(), "v_cache": s["v_cache"].double()}
        out["k_cache"].index_put_(where, turn(s["k"]))
        out["v_cache"].index_put_(where, s["v"].double())
        return out
    if case["op"] == "attend":
        B, H, G, D, page = (case[n] for n in ("B", "H", "G", "D", "page"))
        out = torch.zeros((B, H, D), dtype=torch.float64, device="cuda")
        lse = torch.full((B, H), -math.inf, dtype=torch.float64, device="cuda")
        for b, n in enumerate(s["lengths"].tolist()):
            if n == 0:
                continue
            j = torch.arange(max(0, n - case["window"]) if case["window"] else 0, n, device="cuda")
            where = s["table"][b].long()[j // page], j % page
            k, v = s["k_cache"][where].double(), s["v_cache"][where].double()
            z = torch.einsum("grd,jgd->grj", s["q"][b].double().view(G, H // G, D), k) / math.sqrt(D)
            lse[b] = torch.logsumexp(z, -1).view(H)
            out[b] = torch.einsum("grj,jgd->grd", torch.softmax(z, -1), v).reshape(H, D)
        return {"out": out, "lse": lse}
    x, gamma, Wr = (s[n].double() for n in ("x", "gamma", "Wr"))
    a = x / (x.pow(2).mean(1, keepdim=True) + EPS).sqrt() * gamma
    z = torch.einsum("mk,ek->me", a, Wr)
    experts = torch.argsort(z, dim=1, descending=True, stable=True)[:, :case["k"]]
    w = torch.softmax(z.gather(1, experts), 1)
    y = torch.zeros_like(x)
    for e in experts.unique().tolist():
        m, slot = (experts == e).nonzero(as_tuple=True)
        h = torch.nn.functional.silu(a[m] @ s["Wg"][e].double().t()) * (a[m] @ s["Wu"][e].double().t())
        y[m] += w[m, slot, None] * (h @ s["Wd"][e].double().t())
    return {"y": y, "experts": None, "weights": w}
