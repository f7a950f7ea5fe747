"""What is measured of the operators around a transformer block and at a model's end.

Two operators, each forward and as a training step (forward, then backward):

- ``join``: the norm after a block, its gate, the scaled residual and the norm
  before the next block, in one pass:
      n = norm1(x),  h = residual_scale * residual + block_scale * gate * n,  y = norm2(h)
- ``ce``: softmax cross entropy of a linear head over a large vocabulary, the
  logits never kept:
      z = logit_scale * x W^T,  lse = log sum_v exp(z_v),  loss = lse - z_target
  with loss = lse = 0 (and no gradient) for tokens whose target is negative.

``run`` computes them in plain torch operations in 32 bits, or (``own``) calls
the framework's entry points.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
EPS = 1e-5


# ---------------------------------------------------------------- cases
def _join(name, M, N, norm1, norm2, gates, dtype, train, **more):
    """gates: 0 = no gate, 1 = one gate row for all tokens (a channel scale), G = one gate
    row for each of G equal runs of tokens (a condition for each sample)."""
    return {"name": name, "op": "join", "train": train, "M": M, "N": N, "norm1": norm1, "norm2": norm2,
            "gates": gates, "dtype": dtype, "residual_scale": 1.0, "block_scale": 1.0, **more}


def _ce(name, M, K, V, dtype, train, ignored=0.0, logit_scale=1.0):
    return {"name": name, "op": "ce", "train": train, "M": M, "K": K, "V": V, "dtype": dtype,
            "ignored": ignored, "logit_scale": logit_scale}


def listed():
    return [
        # one token of a decode step between two blocks: latency
        _join("join_token", 1, 8192, "rms", "rms", 1, "bf16", False),
        # a prompt of 8192 tokens through one join (width of the framework's large layers)
        _join("join_prompt", 8192, 8192, "rms", "rms", 1, "bf16", False),
        # a ragged batch at a width that is no multiple of 8, LayerNorm on both sides, no gate
        _join("join_ragged", 513, 14337, "layer", "layer", 0, "f16", False, residual_scale=1.5),
        # a training step of the join at full size
        _join("join_train", 8192, 8192, "rms", "rms", 1, "bf16", True),
        # a training step of a conditioned model: 16 samples of 1000 tokens, a gate row each, LayerNorm
        _join("join_train_samples", 16000, 1152, "layer", "layer", 16, "f16", True),
        # a short fine-tuning batch at an odd width, no norm after the block (a plain pre-norm model)
        _join("join_train_short", 77, 5003, "none", "rms", 0, "bf16", True, block_scale=0.22),
        # the score of one token: the head's weight is read once
        _ce("ce_token", 1, 4096, 131072, "bf16", False),
        # log likelihoods of a few prompts' ends
        _ce("ce_score", 200, 8192, 49152, "f16", False, ignored=0.25),
        # log likelihoods of long documents
        _ce("ce_documents", 8192, 4096, 131072, "bf16", False),
        # a training step of a small model, ragged vocabulary and width
        _ce("ce_train_ragged", 1023, 1000, 32003, "f16", True, ignored=0.1),
        # a training step on few tokens: writing the weight's gradient bounds it
        _ce("ce_train_few", 33, 8192, 65536, "bf16", True),
        # a fine-tuning step, prompts masked out of the loss
        _ce("ce_train", 8192, 4096, 65536, "bf16", True, ignored=0.4),
    ]


def _spread(rng, low, high):
    """A whole number whose logarithm is spread evenly over [low, high]."""
    return min(high, max(low, round(math.exp(rng.uniform(math.log(low), math.log(high + 1))))))


def draw(rng):
    dtype = rng.choice(["bf16", "f16"])
    train = rng.random() < 0.5
    if rng.random() < 0.5:
        while True:
            M, N = _spread(rng, 1, 16384), _spread(rng, 64, 16384)
            N = N if rng.random() < 0.4 else -(-N // 8) * 8
            if M * N <= 1 << 26:
                break
        gates = rng.choice([0, 1, 1, rng.randint(1, 32)])
        if gates > 1:
            M = max(1, M // gates) * gates
        c = _join("", M, N, rng.choice(["none", "layer", "rms", "rms"]), rng.choice(["layer", "rms", "rms"]), gates, dtype,
                  train, residual_scale=rng.choice([1.0, 1.0, 1.25]), block_scale=rng.choice([1.0, 1.0, 0.5]))
    else:
        while True:
            M, K, V = _spread(rng, 1, 8192), _spread(rng, 64, 8192), _spread(rng, 1000, 131072)
            K = K if rng.random() < 0.25 else -(-K // 64) * 64
            if M * K * V <= 1 << 41 and K * V <= 1 << 29:
                break
        c = _ce("", M, K, V, dtype, train, ignored=rng.choice([0.0, 0.0, rng.uniform(0.05, 0.9)]),
                logit_scale=rng.choice([1.0, 1.0, 0.75]))
    del c["name"]
    return c


# --------------------------------------------------------------- inputs
def _ignored(case):
    return min(case["M"] - 1, int(case["ignored"] * case["M"]))


def prepare(case, seed):
    g = torch.Generator("cuda")
    g.manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def normal(*shape, std=1.0, mean=0.0):
        return torch.randn(shape, generator=g, device="cuda") * std + mean

    s = {"case": case}
    if case["op"] == "join":
        M, N = case["M"], case["N"]
        # the residual stream: wider than a block's output, with a few large channels
        wide = 1.0 + 30.0 * (torch.rand(N, generator=g, device="cuda") < 0.002)
        s["x"] = normal(M, N, mean=0.1).to(dt)
        s["residual"] = (normal(M, N, std=2.0) * wide).to(dt)
        for k in ("1", "2"):
            s["gamma" + k] = normal(N, std=0.1, mean=1.0).to(dt) if case["norm" + k] != "none" else None
            s["beta" + k] = normal(N, std=0.1).to(dt) if case["norm" + k] == "layer" else None
        s["gate"] = normal(case["gates"], N, std=0.3, mean=0.5).to(dt) if case["gates"] else None
        if case["train"]:
            s["dy"] = normal(M, N, std=0.1).to(dt)
            s["dh"] = normal(M, N, std=0.1).to(dt)
    else:
        M, K, V = case["M"], case["K"], case["V"]
        s["W"] = torch.empty((V, K), dtype=dt, device="cuda")
        for at in range(0, V, 8192):
            s["W"][at:at + 8192] = normal(min(8192, V - at), K, std=K ** -0.5).to(dt)
        target = torch.randint(0, V, (M,), generator=g, device="cuda")
        # hidden states after a norm; the model has learned some of the targets
        known = 8.0 * torch.rand((M, 1), generator=g, device="cuda")
        s["x"] = (normal(M, K) + known * s["W"][target].float()).to(dt)
        out = torch.randperm(M, generator=g, device="cuda")[:_ignored(case)]
        target[out] = -100
        s["target"] = target
        if case["train"]:
            # the mean over the counted tokens, as a loss-scaled training step has it
            s["dloss"] = torch.full((M,), 1024.0 / (M - _ignored(case)), device="cuda")
    return s


# ------------------------------------------------------------ plain forms
def _norm(kind, v, gamma, beta):
    """(normalized rows, their reciprocal deviation, the output)."""
    if kind == "none":
        return v, None, v
    c = v - v.mean(-1, keepdim=True) if kind == "layer" else v
    r = torch.rsqrt((c * c).mean(-1, keepdim=True) + EPS)
    u = c * r
    o = u * gamma.float()
    return u, r, (o + beta.float() if beta is not None else o)


def _norm_back(kind, u, r, d):
    """The gradient of the normalized rows' input from that of the normalized rows."""
    if kind == "none":
        return d
    t = d - u * (d * u).mean(-1, keepdim=True)
    if kind == "layer":
        t = t - d.mean(-1, keepdim=True)
    return t * r


def _rows(gate, M):
    """A gate row for each token."""
    return gate.float().repeat_interleave(M // gate.shape[0], dim=0) if gate.shape[0] > 1 else gate.float()


def _join_plain(s):
    c = s["case"]
    dt = s["x"].dtype
    u1, r1, n = _norm(c["norm1"], s["x"].float(), s["gamma1"], s["beta1"])
    gate = _rows(s["gate"], c["M"]) if s["gate"] is not None else None
    b = n * c["block_scale"]
    h = s["residual"].float() * c["residual_scale"] + (b * gate if gate is not None else b)
    u2, r2, y = _norm(c["norm2"], h, s["gamma2"], s["beta2"])
    out = {"h": h.to(dt), "y": y.to(dt)}
    if not c["train"]:
        return out
    dy = s["dy"].float()
    dh = s["dh"].float() + _norm_back(c["norm2"], u2, r2, dy * s["gamma2"].float())
    out["dgamma2"] = (dy * u2).sum(0).to(dt)
    if c["norm2"] == "layer":
        out["dbeta2"] = dy.sum(0).to(dt)
    out["dresidual"] = (dh * c["residual_scale"]).to(dt)
    db = dh * c["block_scale"]
    if gate is not None:
        out["dgate"] = (db * n).reshape(c["gates"], -1, c["N"]).sum(1).to(dt)
        db = db * gate
    if c["norm1"] != "none":
        out["dgamma1"] = (db * u1).sum(0).to(dt)
        if c["norm1"] == "layer":
            out["dbeta1"] = db.sum(0).to(dt)
        db = db * s["gamma1"].float()
    out["dx"] = _norm_back(c["norm1"], u1, r1, db).to(dt)
    return out


def _ce_plain(s):
    c = s["case"]
    dt = s["x"].dtype
    target = s["target"]
    counted = target >= 0
    x = torch.where(counted[:, None], s["x"].float(), 0.0)
    W = s["W"].float()
    at = target.clamp(min=0)[:, None]
    z = (x @ W.t()) * c["logit_scale"]
    top = z.max(-1, keepdim=True).values
    p = torch.exp(z - top)
    total = p.sum(-1, keepdim=True)
    lse = (torch.log(total) + top)[:, 0]
    out = {"loss": torch.where(counted, lse - z.gather(1, at)[:, 0], 0.0), "lse": torch.where(counted, lse, 0.0)}
    if not c["train"]:
        return out
    g = torch.where(counted, s["dloss"], 0.0)[:, None] * c["logit_scale"]
    d = p * (g / total)
    d.scatter_add_(1, at, -g)
    out["dx"] = (d @ W).to(dt)
    out["dW"] = (d.t() @ x).to(dt)
    return out


# ------------------------------------------------------- the framework's calls
def _join_own(s):
    import normalization_gemm_row_gb300 as ngr
    c = s["case"]
    kinds = {"none": ngr.NORM_NONE, "layer": ngr.NORM_LAYER, "rms": ngr.NORM_RMS}
    how = dict(gate=s["gate"], norm1=kinds[c["norm1"]], gamma1=s["gamma1"], beta1=s["beta1"], eps1=EPS,
               norm2=kinds[c["norm2"]], gamma2=s["gamma2"], eps2=EPS,
               residual_scale=c["residual_scale"], block_scale=c["block_scale"])
    if not c["train"]:
        h, y = ngr.fused_norm_gate_residual_norm(s["x"], s["residual"], beta2=s["beta2"], **how)
        return {"h": h, "y": y}
    h, y, stats = ngr.fused_norm_gate_residual_norm(s["x"], s["residual"], beta2=s["beta2"], return_stats=True, **how)
    grads = ngr.fused_norm_gate_residual_norm_backward(s["dy"], s["dh"], s["x"], s["residual"], stats, **how)
    out = {"h": h, "y": y}
    for k in ("dgamma2", "dbeta2", "dresidual", "dgate", "dgamma1", "dbeta1", "dx"):
        if grads[k] is not None:
            out[k] = grads[k]
    return out


def _ce_own(s):
    import normalization_gemm_row_gb300 as ngr
    c = s["case"]
    loss, lse = ngr.fused_linear_cross_entropy(s["x"], s["W"], s["target"], logit_scale=c["logit_scale"])
    out = {"loss": loss, "lse": lse}
    if c["train"]:
        out["dx"], out["dW"] = ngr.fused_linear_cross_entropy_backward(
            s["dloss"], lse, s["x"], s["W"], s["target"], logit_scale=c["logit_scale"])
    return out


def run(state):
    if state["case"]["op"] == "join":
        return _join_own(state) if own else _join_plain(state)
    return _ce_own(state) if own else _ce_plain(state)


# ----------------------------------------------------------- work and truth
def work(case):
    if case["op"] == "join":
        M, N = case["M"], case["N"]
        vectors = N * (case["gates"] + sum({"none": 0, "layer": 2, "rms": 1}[case[k]] for k in ("norm1", "norm2")))
        # forward: x, residual in, h, y out; backward: x, residual, dy, dh in, dx, dresidual out
        # (what a training step reads twice, x and the residual, counts once)
        b = 2 * (4 * M * N + vectors)
        f = 20 * M * N
        if case["train"]:
            b += 2 * (4 * M * N + vectors)
            f += 40 * M * N
        return {"bytes": b, "flops": f}
    n, K, V = case["M"] - _ignored(case), case["K"], case["V"]
    b = 2 * K * (V + n) + 16 * case["M"]
    f = 2 * n * K * V
    if case["train"]:
        b += 2 * K * (V + case["M"]) + 4 * case["M"]
        f *= 3
    return {"bytes": b, "flops": f}


def exact(case, seed):
    if case["op"] == "ce" and 8 * case["M"] * case["K"] * case["V"] > 1 << 43:
        return None
    s = prepare(case, seed)
    v = {k: t.double() if torch.is_tensor(t) and t.is_floating_point() else t for k, t in s.items()}
    M = case["M"]
    if case["op"] == "join":
        N = case["N"]

        def core(kind, a):
            """a's rows with the mean taken out (LayerNorm) over sqrt(mean square + eps), and that divisor"""
            if kind == "layer":
                a = a - a.sum(1, keepdim=True) / N
            root = ((a ** 2).sum(1, keepdim=True) / N + EPS).sqrt()
            return (a / root, root) if kind != "none" else (a, None)

        def pull(kind, u, root, d):
            """the vector-Jacobian product of core"""
            if kind == "none":
                return d
            d = d / root - u * ((d * u).sum(1, keepdim=True) / (N * root))
            return d - d.sum(1, keepdim=True) / N if kind == "layer" else d

        def affine(k, u):
            if v["gamma" + k] is None:
                return u
            return u * v["gamma" + k] + (v["beta" + k] if v["beta" + k] is not None else 0.0)

        group = torch.arange(M, device="cuda") // (M // max(1, case["gates"]))
        scale = case["block_scale"] * (v["gate"][group] if v["gate"] is not None else torch.ones((1, 1), dtype=torch.float64, device="cuda"))
        u1, root1 = core(case["norm1"], v["x"])
        n = affine("1", u1)
        h = case["residual_scale"] * v["residual"] + scale * n
        u2, root2 = core(case["norm2"], h)
        out = {"h": h, "y": affine("2", u2)}
        if case["train"]:
            total = v["dh"] + pull(case["norm2"], u2, root2, v["dy"] * v["gamma2"])
            out["dgamma2"] = torch.einsum("mn,mn->n", v["dy"], u2)
            if v["beta2"] is not None:
                out["dbeta2"] = v["dy"].sum(0)
            out["dresidual"] = case["residual_scale"] * total
            if v["gate"] is not None:
                out["dgate"] = torch.zeros_like(v["gate"]).index_add_(0, group, case["block_scale"] * total * n)
            dn = scale * total
            if v["gamma1"] is not None:
                out["dgamma1"] = torch.einsum("mn,mn->n", dn, u1)
                if v["beta1"] is not None:
                    out["dbeta1"] = dn.sum(0)
                dn = dn * v["gamma1"]
            out["dx"] = pull(case["norm1"], u1, root1, dn)
        return out
    keep = (v["target"] >= 0).nonzero()[:, 0]
    t = v["target"][keep]
    x = v["x"][keep]
    a = case["logit_scale"]
    out = {"loss": torch.zeros(M, dtype=torch.float64, device="cuda"), "lse": torch.zeros(M, dtype=torch.float64, device="cuda")}
    if case["train"]:
        out["dx"], out["dW"] = torch.zeros_like(v["x"]), torch.zeros_like(v["W"])
    for at in range(0, len(keep), 1024):
        rows, lab, xs = keep[at:at + 1024], t[at:at + 1024], x[at:at + 1024]
        z = a * torch.einsum("mk,vk->mv", xs, v["W"])
        lse = torch.logsumexp(z, 1)
        out["lse"][rows] = lse
        out["loss"][rows] = lse - z[torch.arange(len(rows), device="cuda"), lab]
        if case["train"]:
            d = torch.exp(z - lse[:, None])
            d[torch.arange(len(rows), device="cuda"), lab] -= 1.0
            d *= a * v["dloss"][rows][:, None]
            out["dx"][rows] = torch.einsum("mv,vk->mk", d, v["W"])
            out["dW"] += torch.einsum("mv,mk->vk", d, xs)
    return out
