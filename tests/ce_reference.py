"""The linear cross entropy and its gradient in float64 on the CPU, and how
far a correct computation of this precision may be from it."""
import torch

U = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}       # half a step, relative
TINY = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}


def case(M, K, V, dtype, seed, ignored=0.0, peaked=6.0, spread=1.0):
    g = torch.Generator("cpu")
    g.manual_seed(seed)
    W = (torch.randn((V, K), generator=g) * K ** -0.5 * spread).to(dtype)
    target = torch.randint(0, V, (M,), generator=g)
    x = torch.randn((M, K), generator=g) + peaked * torch.rand((M, 1), generator=g) * W[target].float()
    if ignored:
        out = torch.rand(M, generator=g) < ignored
        target[out] = torch.randint(-100, 0, (int(out.sum()),), generator=g)
    return {"x": x.to(dtype), "W": W, "target": target, "dloss": torch.rand(M, generator=g) * 0.1 + 0.01,
            "dlse": torch.randn(M, generator=g) * 0.02}


def reference(d, scale=1.0, dloss=None, dlse=None):
    """Values and tolerances: loss, lse (absolute), dx, dW."""
    dtype = d["x"].dtype
    u = U[dtype]
    t = d["target"]
    on = t >= 0
    x = torch.where(on[:, None], d["x"].double(), 0.0)
    W = d["W"].double()
    M, K = x.shape
    V = W.shape[0]
    z = scale * x @ W.T
    at = t.clamp(min=0)[:, None]
    lse = torch.logsumexp(z, 1)
    zt = z.gather(1, at)[:, 0]
    val = {"loss": torch.where(on, lse - zt, 0.0), "lse": torch.where(on, lse, 0.0)}
    # A logit is an FP32 sum of K exact products: each of its K / 16 tensor
    # core steps (and the sums inside one, taken as 16 more) may lose a whole
    # step of 2^-23 of the running sum, which is at most the sum of sizes.
    size = abs(scale) * (x.abs() @ W.abs().T)
    ez = (K / 16 + 16) * 2.0 ** -23 * size
    # lse: the largest logit error, and a sum over the vocabulary of
    # exponentials good to 2^-21 in up to 64 additions a thread and 12 levels.
    el = ez.max(1).values + 80 * 2.0 ** -23 + 2.0 ** -22 * lse.abs()
    tol = {"lse": el, "loss": el + ez.gather(1, at)[:, 0] + 2.0 ** -23 * (lse.abs() + zt.abs())}
    if dloss is None and dlse is None:
        return val, tol
    g = torch.where(on, dloss.double() if dloss is not None else torch.zeros(M, dtype=torch.float64), 0.0)[:, None]
    gl = torch.where(on, dlse.double() if dlse is not None else torch.zeros(M, dtype=torch.float64), 0.0)[:, None]
    p = torch.exp(z - lse[:, None])
    hot = torch.zeros_like(z).scatter_(1, at, 1.0)
    dz = scale * ((g + gl) * p - g * hot)
    val["dx"], val["dW"] = dz @ W, dz.T @ x
    # dz: p's error (logit and lse), then one rounding to the 16-bit type
    # (below its normal range a fixed step: the scaled weights reach 2^13, so
    # that step is 2^-25 2^-13 of the largest weight)
    # p below 2^-126, FP32's smallest normal number, may be taken as 0: off by
    # less than 2^-126 of the weight (it shows in bf16, whose range goes there).
    most = (abs(scale) * torch.maximum(g.abs(), (g + gl).abs())).max()
    edz = abs(scale) * (g + gl).abs() * (p * (ez + el[:, None] + 2.0 ** -20) + 2.0 ** -126) + u * dz.abs() * 1.01 + \
        abs(scale) * g.abs() * hot * 2.0 ** -23 + (2.0 ** -37 * most if dtype == torch.float16 else 0.0)
    acc = lambda n: (n / 16 + 80) * 2.0 ** -23      # FP32 accumulation over n terms
    tol["dx"] = edz @ W.abs() + acc(V) * (dz.abs() @ W.abs()) + u * val["dx"].abs() + TINY[dtype]
    tol["dW"] = edz.T @ x.abs() + acc(M) * (dz.abs().T @ x.abs()) + u * val["dW"].abs() + TINY[dtype]
    return val, tol


def check(got, val, tol, what):
    got = got.double().cpu()
    assert got.shape == val.shape, what
    assert torch.isfinite(got).all(), f"{what}: not finite"
    err = (got - val).abs()
    assert (err <= tol + 1e-300).all(), (f"{what}: {(err > tol).sum().item()} of {err.numel()} out, worst "
                                         f"{(err / (tol + 1e-300)).max().item():.2f} times the tolerance, "
                                         f"max {err.max().item():.3e}")
    return (err / (tol + 1e-300)).max().item() if err.numel() else 0.0
