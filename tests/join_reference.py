"""The block join and its gradient in float64 on the CPU, and how far a
correct FP32 computation may be from it."""
import torch

U = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}      # half a step, relative
TINY = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}  # half a step among the subnormals


def case(M, N, norm1, norm2, gates, dtype, seed, residual=True, mean=0.3, spread=1.0):
    g = torch.Generator("cpu")
    g.manual_seed(seed)

    def normal(*shape, std=1.0, mean=0.0):
        return (torch.randn(shape, generator=g) * std + mean).to(dtype)

    d = {"x": normal(M, N, std=spread, mean=mean), "residual": normal(M, N, std=2.0) if residual else None,
         "gate": normal(gates, N, std=0.3, mean=0.5) if gates else None,
         "gamma1": normal(N, std=0.2, mean=1.0) if norm1 else None,
         "beta1": normal(N, std=0.2) if norm1 == 1 else None,
         "gamma2": normal(N, std=0.2, mean=1.0) if norm2 else None,
         "beta2": normal(N, std=0.2) if norm2 == 1 else None,
         "dy": normal(M, N) if norm2 else None, "dh": normal(M, N)}
    return d


def _core(kind, v, eps):
    if kind == 0:
        return v
    if kind == 1:
        v = v - v.mean(-1, keepdim=True)
    return v / torch.sqrt((v * v).mean(-1, keepdim=True) + eps)


def forward(d, norm1, norm2, eps=1e-5, a=1.0, s=1.0):
    """h, y, n as differentiable functions of the float64 tensors of d."""
    M, N = d["x"].shape
    n = _core(norm1, d["x"], eps)
    if norm1:
        n = n * d["gamma1"]
        if norm1 == 1:
            n = n + d["beta1"]
    b = s * n
    if d["gate"] is not None:
        b = b * d["gate"].repeat_interleave(M // d["gate"].shape[0], dim=0)
    h = b if d["residual"] is None else a * d["residual"] + b
    y = None
    if norm2:
        y = _core(norm2, h, eps) * d["gamma2"]
        if norm2 == 1:
            y = y + d["beta2"]
    return h, y


def reference(d, norm1, norm2, eps=1e-5, a=1.0, s=1.0):
    """(values, magnitudes): the outputs and gradients by autograd in
    float64, and for each the sum of the sizes of the terms it is made of."""
    w = {k: (v.double().requires_grad_(k not in ("dy", "dh")) if v is not None else None) for k, v in d.items()}
    h, y = forward(w, norm1, norm2, eps, a, s)
    loss = (h * w["dh"]).sum() if w["dh"] is not None else 0.0
    if norm2 and w["dy"] is not None:
        loss = loss + (y * w["dy"]).sum()
    names = [k for k in ("x", "residual", "gate", "gamma1", "beta1", "gamma2", "beta2") if w[k] is not None]
    # (an input that the loss does not reach has gradient zero)
    grads = torch.autograd.grad(loss, [w[k] for k in names], allow_unused=True)
    val = {"h": h.detach(), "y": y.detach() if y is not None else None}
    for k, gr in zip(names, grads):
        val["d" + k] = gr if gr is not None else torch.zeros_like(w[k])

    with torch.no_grad():
        M, N = d["x"].shape
        v = {k: (t.double() if t is not None else None) for k, t in d.items()}
        one = torch.ones((1, N), dtype=torch.float64)
        rows = v["gate"].repeat_interleave(M // v["gate"].shape[0], dim=0) if v["gate"] is not None else one

        def stats(kind, t):
            mu = t.mean(-1, keepdim=True) if kind == 1 else torch.zeros((M, 1), dtype=torch.float64)
            rs = 1.0 / torch.sqrt(((t - mu) ** 2).mean(-1, keepdim=True) + eps) if kind else torch.ones((M, 1), dtype=torch.float64)
            return mu, rs

        mu1, rs1 = stats(norm1, v["x"])
        u1 = (v["x"].abs() + mu1.abs()) * rs1
        g1 = v["gamma1"].abs() if norm1 else one
        n = u1 * g1 + (v["beta1"].abs() if norm1 == 1 else 0.0)
        gs = abs(s) * rows.abs()
        hm = gs * n + (abs(a) * v["residual"].abs() if v["residual"] is not None else 0.0)
        mu2, rs2 = stats(norm2, val["h"])
        u2 = (hm + mu2.abs()) * rs2 if norm2 else torch.zeros_like(hm)
        # the variance's own error moves u2 as a whole
        u2 = u2 * (1.0 + (hm * hm).mean(-1, keepdim=True) * rs2 * rs2) if norm2 else u2
        g2 = v["gamma2"].abs() if norm2 else one
        mag = {"h": hm, "y": u2 * g2 + (v["beta2"].abs() if norm2 == 1 else 0.0)}
        dy = v["dy"].abs() if norm2 and v["dy"] is not None else torch.zeros_like(hm)
        q = dy * g2
        D = v["dh"].abs() if v["dh"] is not None else torch.zeros_like(hm)
        if norm2:
            D = D + rs2 * (q + q.mean(-1, keepdim=True) + u2 * (q * u2).mean(-1, keepdim=True))
        mag["dresidual"] = abs(a) * D
        if v["gate"] is not None:
            mag["dgate"] = (abs(s) * n * D).reshape(v["gate"].shape[0], -1, N).sum(1)
        dn = gs * D
        mag["dgamma1"] = (dn * u1).sum(0)
        mag["dbeta1"] = dn.sum(0)
        mag["dgamma2"] = (dy * u2).sum(0)
        mag["dbeta2"] = dy.sum(0)
        w1 = dn * g1
        mag["dx"] = rs1 * (w1 + w1.mean(-1, keepdim=True) + u1 * (w1 * u1).mean(-1, keepdim=True)) if norm1 else w1
    return val, mag


# FP32 slack relative to the sizes of the terms: a term passes through fewer
# than 64 FP32 operations of half a step 2^-24 each, and every sum is a tree
# of at most 64 sequential additions and 12 levels over terms counted with
# their sizes: (64 + 64) 2^-24 = 2^-17.
SLACK = 2.0 ** -17


def check(got, val, mag, dtype, what):
    got = got.double().cpu()
    assert got.shape == val.shape, what
    assert torch.isfinite(got).all(), f"{what}: not finite"
    tol = U[dtype] * val.abs() + (1 + U[dtype]) * SLACK * mag + TINY[dtype]
    over = (got - val).abs() - tol
    assert (over <= 0).all(), (f"{what}: {(over > 0).sum().item()} of {val.numel()} out, worst "
                               f"{((got - val).abs() / tol).max().item():.2f} times the tolerance")
