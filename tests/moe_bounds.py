"""How far the mixture-of-experts layer may be from its formula in float64 when
its products take a and h in two parts of the inputs' type, as it says: a
bound on every error's size, without the single roundings that
moe_reference.py admits."""
import torch

from moe_reference import TINY, U, case as make_case, chain as router_chain, normalized, separate

FLOOR = {torch.float16: 2.0 ** -28, torch.bfloat16: 2.0 ** -126}


def two_parts(x, dtype):
    """A value rounded and what that left out, rounded: half a step of half a step, or the small end."""
    return torch.clamp(U[dtype] ** 2 * x.abs(), min=FLOOR[dtype])


def chain(n):
    """A sum of n products, relative to the sum S of their sizes.  A matrix instruction adds 16 of them to what is there:
    it cuts the 17 addends off at 2^-25 of the largest's power of two and their sum at 2^-23, together below 2^-20.5 of
    the sizes so far, on average of S / 2.  A row's parts of at least sqrt(n / 64) steps are joined by as many rounding
    additions; 16 more for the two columns, tokens' sums and the like."""
    return n / 16 * 2.0 ** -21.5 + ((n / 64) ** 0.5 + 16) * 2.0 ** -24


def reference(d, top_k, norm=2, eps=1e-5, renormalize=True):
    """(y, experts, weights, tolerance of y, of the weights (relative)), as moe_reference.reference."""
    dtype = d["x"].dtype
    a = normalized(d, norm, eps)
    M, K = a.shape
    F = d["Wg"].shape[1]
    few = 2.0 ** -20      # a few steps of FP32: the norm; SiLU
    z = a @ d["Wr"].double().t()
    order = torch.argsort(z, dim=1, descending=True, stable=True)[:, :top_k]
    p = torch.softmax(z, 1).gather(1, order)
    if renormalize:
        p = p / p.sum(1, keepdim=True)
    dz = ((router_chain(K) + few) * (a.abs() @ d["Wr"].double().abs().t())).max(1, keepdim=True).values
    tol_p = 2 * dz + few
    da = two_parts(a, dtype) + (few * a.abs() if norm else 0.0)
    y, tol = (torch.zeros((M, K), dtype=torch.float64) for _ in range(2))
    for e in order.unique().tolist():
        m, s = (order == e).nonzero(as_tuple=True)
        wg, wu, wd = (d[n][e].double() for n in ("Wg", "Wu", "Wd"))
        am, pm = a[m], p[m, s][:, None]
        gate, up = am @ wg.t(), am @ wu.t()
        silu = gate * torch.sigmoid(gate)
        dg, du = (da[m] @ w.abs().t() + chain(K) * (am.abs() @ w.abs().t()) for w in (wg, wu))
        h = pm * silu * up
        # SiLU's slope is below 1.1
        dh = pm * (1.1 * dg * up.abs() + silu.abs() * du + 1.1 * dg * du) + (few + tol_p[m]) * h.abs() + two_parts(h, dtype)
        y[m] += h @ wd.t()
        tol[m] += (dh + chain(F * top_k) * h.abs()) @ wd.abs().t()
    return y, order, p, tol + U[dtype] * y.abs() + TINY[dtype], tol_p


# (M, K, F, E, top_k): ordinary sizes, widths that end inside a step or off the 16-byte boundary, rows of down's result
# that many workers share
CASES = [(5, 256, 192, 8, 2), (6, 64, 40, 33, 5), (32, 61, 45, 5, 3), (7, 65, 63, 6, 2), (4, 1000, 2001, 5, 2), (4, 1001, 500, 5, 2),
         (19, 130, 2500, 8, 4), (4, 4100, 72, 5, 2), (4, 8200, 40, 5, 2), (29, 40, 6001, 20, 5), (2, 40, 6000, 16, 4)]


def case(M, K, F, E, top_k, dtype, norm=2):
    """Inputs whose last columns weigh the more, so that one that is lost shows: their share of the results is about 8 /
    sqrt(K) and 8 / sqrt(F) of them."""
    d = make_case(M, K, F, E, dtype, seed=M + K + F, norm=norm)
    d["x" if norm == 0 else "gamma"][..., -1] *= 8
    d["Wd"][..., -1] *= 8
    return separate(d, top_k, norm)


def sparse_case(M, K, F, E, top_k, dtype, norm=2):
    """Inputs of which three columns of K and of F count, the first, a middle one and the last: nothing averages out, so
    that a single rounding of a or of h shows."""
    d = make_case(M, K, F, E, dtype, seed=2 * (M + K + F) + norm, norm=norm)
    few_k, few_f = ([0, n // 2, n - 1] for n in (K, F))
    x, wd = torch.zeros_like(d["x"]), torch.zeros_like(d["Wd"])
    x[:, few_k] = d["x"][:, few_k] * (1.0 if norm else K ** 0.5)
    wd[..., few_f] = d["Wd"][..., few_f]
    d["x"], d["Wd"] = x, wd
    return separate(d, top_k, norm)
