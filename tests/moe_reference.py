"""The mixture-of-experts layer in float64 on the CPU, and how far a correct
computation with its roundings may be from it."""
import math

import torch

U = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}      # half a step, relative
TINY = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}  # half a step among the subnormals


def case(M, K, F, E, dtype, seed=0, norm=2):
    g = torch.Generator("cpu")
    g.manual_seed(seed)

    def normal(*shape, std=1.0, mean=0.0):
        return (torch.randn(shape, generator=g) * std + mean).to(dtype)

    return {"x": normal(M, K, mean=0.1), "Wr": normal(E, K, std=1.5 * K ** -0.5), "Wg": normal(E, F, K, std=K ** -0.5),
            "Wu": normal(E, F, K, std=K ** -0.5), "Wd": normal(E, K, F, std=F ** -0.5),
            "gamma": normal(K, std=0.2, mean=1.0) if norm else None, "beta": normal(K, std=0.2) if norm == 1 else None}


def normalized(d, norm, eps):
    x = d["x"].double()
    if norm == 1:
        x = x - x.mean(-1, keepdim=True)
    if norm:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * d["gamma"].double()
    return x + d["beta"].double() if norm == 1 else x


def chain(n):
    """FP32 sums of n terms in the order of the matrix instructions: chains of
    n / 64 + 64 additions, each off by at most a step 2^-23 of the terms' sizes."""
    return (n / 64 + 64) * 2.0 ** -23


def reference(d, top_k, norm=2, eps=1e-5, renormalize=True):
    """(y, experts, weights, tolerance of y, of the weights (relative)).

    Roundings of a and of h to the 16-bit type are independent, zero in the
    mean and at most half a step: a sum of such errors c_i stays within 8
    sqrt(sum c_i^2) but for a chance of 2 exp(-32) (Hoeffding)."""
    dtype = d["x"].dtype
    u, tiny = U[dtype], TINY[dtype]
    a = normalized(d, norm, eps)
    M, K = a.shape
    E, F, _ = d["Wg"].shape
    z = a @ d["Wr"].double().t()
    order = torch.argsort(z, dim=1, descending=True, stable=True)[:, :top_k]
    p = torch.softmax(z, 1).gather(1, order)
    if renormalize:
        p = p / p.sum(1, keepdim=True)
    # FP32 logits: the norm's few steps and the sum's
    dz = ((chain(K) + 2.0 ** -20) * (a.abs() @ d["Wr"].double().abs().t())).max(1, keepdim=True).values
    tol_p = 2 * dz + 2.0 ** -20
    y = torch.zeros((M, K), dtype=torch.float64)
    square, flat = torch.zeros_like(y), torch.zeros_like(y)
    for e in order.unique().tolist():
        m, s = (order == e).nonzero(as_tuple=True)
        wg, wu, wd = (d[n][e].double() for n in ("Wg", "Wu", "Wd"))
        am, pm = a[m], p[m, s][:, None]
        gate, up = am @ wg.t(), am @ wu.t()
        silu = gate * torch.sigmoid(gate)

        def off(w):
            return 8 * torch.sqrt((u * am) ** 2 @ (w * w).t()) + (chain(K) + 2.0 ** -20) * (am.abs() @ w.abs().t())

        dg, du = off(wg), off(wu)
        h = pm * silu * up
        # SiLU's slope is below 1.1
        dh = pm * (1.1 * dg * up.abs() + silu.abs() * du + 1.1 * dg * du) + 8 * (u * h.abs() + tiny)
        y[m] += h @ wd.t()
        square[m] += dh ** 2 @ (wd * wd).t()
        flat[m] += (chain(F * top_k) + tol_p[m] + 2.0 ** -20) * (h.abs() @ wd.abs().t())
    tol = torch.sqrt(square) + flat + u * y.abs() + tiny
    return y, order, p, tol, tol_p


def check(got, want, what=""):
    y, experts, weights = (t.cpu() for t in got)
    vy, ve, vw, tol, tol_p = want
    assert torch.equal(experts.long(), ve), f"{what}: experts"
    assert ((weights.double() - vw).abs() <= tol_p * vw).all(), f"{what}: weights"
    assert torch.isfinite(y).all(), f"{what}: not finite"
    r = (y.double() - vy).abs() / tol
    assert (r <= 1).all(), f"{what}: y worst {r.max().item():.2f} times the tolerance"
    return r.max().item()


def apart(d, top_k, norm=2, eps=1e-5):
    """Whether no token's choice hangs on FP32 rounding."""
    a = normalized(d, norm, eps)
    z = torch.sort(a @ d["Wr"].double().t(), dim=1, descending=True).values[:, :top_k + 1]
    return z.shape[1] < 2 or (z[:, :-1] - z[:, 1:]).min().item() > 1e-5


def separate(d, top_k, norm=2, eps=1e-5):
    """d with the router's rows nudged (by scaling expert e's by 1 + e / 64) until the choices stand apart."""
    for _ in range(8):
        if apart(d, top_k, norm, eps):
            return d
        e = torch.arange(d["Wr"].shape[0], dtype=torch.float64)[:, None]
        d["Wr"] = (d["Wr"].double() * (1 + e / 64)).to(d["Wr"].dtype)
    raise AssertionError("choices too close")


assert math.isclose(chain(64), 65 * 2.0 ** -23)
