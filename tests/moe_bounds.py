"""How far the mixture-of-experts layer may be from its formula in float64 when
its products take a and h in two parts of the inputs' type, as it says: a
bound on every error's size, without the single roundings that
moe_reference.py admits."""
import torch

from moe_reference import TINY, U, chain as router_chain, normalized

FLOOR = {torch.float16: 2.0 ** -28, torch.bfloat16: 2.0 ** -126}


def two_parts(x, dtype):
    """A value rounded and what that left out, rounded: half a step of half a step, or the small end."""
    return torch.clamp(U[dtype] ** 2 * x.abs(), min=FLOOR[dtype])


def chain(n):
    """A sum of n products in FP32, 16 at a time, relative to the sum S of their sizes.  An addition of 16 is off by at
    most 2^-22 of what it has so far, on average S / 2: n / 16 of them 2^-23 n / 16.  A row's parts of at least sqrt(n /
    64) steps are joined by as many additions; 16 more for the two columns, tokens' sums and the like."""
    return (n / 16 + (n / 64) ** 0.5 + 16) * 2.0 ** -23


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
