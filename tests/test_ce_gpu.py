"""GPU parity of the linear cross entropy and its gradient against the
formulas in float64.  The tolerance is derived in ce_reference.py."""
import pytest
import torch

import normalization_gemm_row_gb300 as ngr
from normalization_gemm_row_gb300 import binding as B
import ce_reference as R

pytestmark = pytest.mark.gpu
DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _built():
    ngr.build()
    torch.cuda.init()


def cuda(d):
    return {k: v.cuda() for k, v in d.items()}


def run(d, scale=1.0, dlse=False):
    c = cuda(d)
    loss, lse = ngr.fused_linear_cross_entropy(c["x"], c["W"], c["target"], logit_scale=scale)
    dx, dW = ngr.fused_linear_cross_entropy_backward(c["dloss"], lse, c["x"], c["W"], c["target"], logit_scale=scale,
                                                     dlse=c["dlse"] if dlse else None)
    return {"loss": loss, "lse": lse, "dx": dx, "dW": dW}


def compare(d, what, scale=1.0, dlse=False):
    got = run(d, scale, dlse)
    val, tol = R.reference(d, scale, d["dloss"], d["dlse"] if dlse else None)
    for k in ("loss", "lse", "dx", "dW"):
        R.check(got[k], val[k], tol[k], f"{what} {k}")
    off = d["target"] < 0
    assert (got["loss"].cpu()[off] == 0).all() and (got["lse"].cpu()[off] == 0).all() and (got["dx"].cpu()[off] == 0).all()
    return got


# One token, one entry, tiles' edges, ragged rows, widths and vocabularies,
# several row tiles, ranges of the vocabulary with their own sums.
SHAPES = [(1, 64, 1), (1, 8, 2), (1, 256, 1000), (2, 72, 129), (17, 64, 255), (33, 128, 256), (128, 64, 257),
          (129, 200, 500), (255, 320, 640), (256, 256, 1024), (257, 512, 513), (300, 1000, 2003), (700, 96, 5000),
          (64, 1024, 9000), (1025, 64, 300)]


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("M,K,V", SHAPES)
def test_sizes(M, K, V, dtype):
    compare(R.case(M, K, V, DTYPES[dtype], seed=M + K + V), f"{M}x{K}x{V}")


@pytest.mark.parametrize("K", [1, 3, 7, 63, 65, 130, 1001])
def test_any_width(K):
    """Widths that are no multiple of 8: W is copied with padded rows."""
    for dtype in DTYPES.values():
        compare(R.case(37, K, 301, dtype, seed=K), f"K={K}", scale=0.7)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("M,ignored", [(1, 1.0), (50, 0.5), (300, 0.9), (600, 0.3), (600, 1.0)])
def test_masked_tokens(M, ignored, dtype):
    """Masked tokens may hold anything: the result is that of the others."""
    d = R.case(M, 136, 700, DTYPES[dtype], seed=M + int(10 * ignored), ignored=ignored)
    off = d["target"] < 0
    d["x"][off] = float("nan")
    d["dloss"][off] = float("inf")
    d["x"][off.nonzero()[::2, 0]] = float("inf")
    got = compare(d, f"{M} tokens, {ignored} masked", dlse=False)
    if off.all():
        assert (got["dW"] == 0).all()


def test_penalty_on_lse_and_scale():
    d = R.case(200, 256, 1500, torch.bfloat16, seed=3, ignored=0.2)
    for scale in (1.0, 0.25, -0.5, 0.0):
        compare(d, f"scale {scale}", scale=scale, dlse=True)
    c = cuda(d)
    _, lse = ngr.fused_linear_cross_entropy(c["x"], c["W"], c["target"])
    dx, dW = ngr.fused_linear_cross_entropy_backward(None, lse, c["x"], c["W"], c["target"], dlse=c["dlse"])
    val, tol = R.reference(d, 1.0, None, d["dlse"])
    R.check(dx, val["dx"], tol["dx"], "dlse alone dx")
    R.check(dW, val["dW"], tol["dW"], "dlse alone dW")


@pytest.mark.parametrize("size", [1e-30, 1e-9, 1.0, 1e6])
def test_weights_of_any_size(size):
    """fp16's range holds p times the weight at any size of the weights."""
    d = R.case(60, 64, 900, torch.bfloat16, seed=9)
    d["dloss"] = d["dloss"] * size
    compare(d, f"dloss about {size}")
    if 1e-9 < size < 1e6:
        h = R.case(60, 64, 900, torch.float16, seed=9)
        h["dloss"] = h["dloss"] * size
        compare(h, f"fp16 dloss about {size}")


def test_large_logits():
    """Logits of hundreds: the softmax is a step, nothing overflows."""
    for dtype in DTYPES.values():
        d = R.case(40, 256, 777, dtype, seed=4, peaked=0.0, spread=40.0)
        compare(d, "large logits")


@pytest.mark.parametrize("dtype", list(DTYPES))
def test_infinite_logits(dtype):
    """An entry of W that overflowed: +inf or -inf in one logit of each token,
    and what the formula makes of them.  A token with +inf has lse = loss =
    inf and gives the other entries no gradient; where the formula has no
    value (inf - inf) there is NaN, and nowhere else."""
    d = R.case(70, 64, 600, DTYPES[dtype], seed=8, peaked=0.0)
    d["x"][:, 0] = 1.0 - 2.0 * (torch.arange(70) % 2)
    d["target"][d["target"] == 300] = 301
    plain = {**d, "W": d["W"].clone()}
    d["W"][300, 0] = float("inf")
    plain["W"][300] = 0.0
    got = run(d)
    val, _ = R.reference(d, 1.0, d["dloss"])
    up = torch.arange(70) % 2 == 0
    assert torch.isinf(val["lse"][up]).all() and torch.isfinite(val["lse"][~up]).all()
    for k in ("loss", "lse", "dx", "dW"):
        a, b = got[k].double().cpu(), val[k]
        assert torch.equal(torch.isnan(a), torch.isnan(b)) and torch.equal(torch.isinf(a), torch.isinf(b)), k
    # the tolerance of the tokens with -inf: that of a logit of 0 there, which
    # has no smaller sums
    _, tol = R.reference(plain, 1.0, d["dloss"])
    for k in ("loss", "lse"):
        R.check(got[k].cpu()[~up], val[k][~up], tol[k][~up], k)


def test_one_output_only():
    d = R.case(90, 128, 400, torch.float16, seed=5)
    full = run(d)
    c = cuda(d)
    a = ngr.fused_linear_cross_entropy_backward(c["dloss"], full["lse"], c["x"], c["W"], c["target"], need_dW=False)
    b = ngr.fused_linear_cross_entropy_backward(c["dloss"], full["lse"], c["x"], c["W"], c["target"], need_dx=False)
    assert a[1] is None and b[0] is None
    assert torch.equal(a[0], full["dx"]) and torch.equal(b[1], full["dW"])


def test_target_outside_the_vocabulary_is_reported():
    d = R.case(20, 64, 100, torch.bfloat16, seed=6)
    d["target"][7] = 100
    d["target"][9] = 1 << 40
    c = cuda(d)
    n = B.ngr_linear_cross_entropy_workspace_bytes(0, 20, 64, 100)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    loss, lse = ngr.fused_linear_cross_entropy(c["x"], c["W"], c["target"], workspace=ws)
    assert B.ngr_workspace_error(ws.data_ptr(), torch.cuda.current_stream().cuda_stream) == -9
    assert B.ngr_workspace_error(ws.data_ptr(), torch.cuda.current_stream().cuda_stream) == 0
    d["target"][7] = d["target"][9] = -1
    val, tol = R.reference(d)
    R.check(loss, val["loss"], tol["loss"], "the other tokens")


def test_pieces_of_the_vocabulary():
    """More tokens than one piece of 256 MB holds of the whole vocabulary:
    dx adds up over the pieces."""
    M, K, V = 9000, 64, 18000
    d = R.case(M, K, V, torch.bfloat16, seed=7, ignored=0.1)
    got = run(d)
    rows = torch.randperm(M, generator=torch.Generator().manual_seed(1))[:300]
    part = {k: (v[rows] if k != "W" else v) for k, v in d.items()}
    val, tol = R.reference(part, 1.0, part["dloss"])
    for k in ("loss", "lse", "dx"):
        R.check(got[k].cpu()[rows], val[k], tol[k], k)
    # dW: some rows of it, from every token (float64 on the GPU for the sums)
    c = cuda(d)
    on = c["target"] >= 0
    x = torch.where(on[:, None], c["x"].double(), 0.0)
    z = x @ c["W"].double().T
    p = torch.exp(z - torch.logsumexp(z, 1, keepdim=True)) * torch.where(on, c["dloss"].double(), 0.0)[:, None]
    p[torch.arange(M, device="cuda"), c["target"].clamp(min=0)] -= torch.where(on, c["dloss"].double(), 0.0)
    want, size = p.T @ x, p.abs().T @ x.abs()
    err = (got["dW"].double() - want).abs()
    assert (err <= 2.0 ** -8 * want.abs() + (1.1 * 2.0 ** -8 + 2.0 ** -14) * size + 1e-30).all()


@pytest.mark.parametrize("K", [64, 61])
def test_any_even_address(K):
    """x, dx and dW one element off a 16-byte boundary (and W where its rows
    are copied anyway)."""
    M, V = 30, 333
    d = R.case(M, K, V, torch.float16, seed=K)
    off = lambda t: torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")[1:].view(t.shape).copy_(t)
    x, W = off(d["x"]), (off(d["W"]) if K % 8 else d["W"].cuda())
    t, g = d["target"].cuda(), d["dloss"].cuda()
    loss, lse = ngr.fused_linear_cross_entropy(x, W, t)
    dx, dW = off(torch.zeros_like(x)), off(torch.zeros_like(W))
    n = B.ngr_linear_cross_entropy_workspace_bytes(1, M, K, V)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    s = torch.cuda.current_stream().cuda_stream
    assert B.ngr_fused_linear_cross_entropy_backward(g.data_ptr(), None, lse.data_ptr(), x.data_ptr(), W.data_ptr(),
                                                     t.data_ptr(), 1.0, M, K, V, 0, dx.data_ptr(), dW.data_ptr(),
                                                     ws.data_ptr(), n, s) == 0
    val, tol = R.reference(d, 1.0, d["dloss"])
    for got, k in ((loss, "loss"), (dx, "dx"), (dW, "dW")):
        R.check(got, val[k], tol[k], k)


@pytest.mark.parametrize("K", [264, 131])
def test_same_call_same_bits_and_nothing_else_written(K):
    M, V = 140, 1030
    d = R.case(M, K, V, torch.bfloat16, seed=8, ignored=0.2)
    a, b = run(d), run(d)
    for k in a:
        assert torch.equal(a[k], b[k]), k
    # outputs and workspace inside larger buffers
    c = cuda(d)
    s = torch.cuda.current_stream().cuda_stream
    n = [B.ngr_linear_cross_entropy_workspace_bytes(i, M, K, V) for i in (0, 1)]
    ws = torch.full((max(n) + 512,), 0x5A, dtype=torch.uint8, device="cuda")
    vec = torch.full((2, M + 8), 7.0, device="cuda")
    dx = torch.full((M + 3, K), 7.0, dtype=torch.bfloat16, device="cuda")
    dW = torch.full((V + 3, K), 7.0, dtype=torch.bfloat16, device="cuda")
    p = lambda t: t.data_ptr()
    assert B.ngr_fused_linear_cross_entropy(p(c["x"]), p(c["W"]), p(c["target"]), 1.0, M, K, V, 1, p(vec[0]), p(vec[1]),
                                            p(ws), n[0], s) == 0
    torch.cuda.synchronize()
    assert (ws[n[0]:] == 0x5A).all()
    assert B.ngr_fused_linear_cross_entropy_backward(p(c["dloss"]), None, p(vec[1]), p(c["x"]), p(c["W"]), p(c["target"]),
                                                     1.0, M, K, V, 1, p(dx), p(dW), p(ws), n[1], s) == 0
    torch.cuda.synchronize()
    assert (ws[n[1]:] == 0x5A).all() and (vec[:, M:] == 7).all() and (dx[M:] == 7).all() and (dW[V:] == 7).all()
    assert torch.equal(vec[0, :M], a["loss"]) and torch.equal(dx[:M], a["dx"]) and torch.equal(dW[:V], a["dW"])


def test_empty_batch():
    W = torch.randn(50, 64, device="cuda").half()
    x = torch.empty(0, 64, dtype=torch.float16, device="cuda")
    t = torch.empty(0, dtype=torch.int64, device="cuda")
    loss, lse = ngr.fused_linear_cross_entropy(x, W, t)
    dx, dW = ngr.fused_linear_cross_entropy_backward(loss, lse, x, W, t)
    assert loss.shape == (0,) and dx.shape == (0, 64) and (dW == 0).all()


def test_captured_and_on_another_stream():
    d = R.case(270, 192, 1200, torch.bfloat16, seed=10, ignored=0.3)
    want = run(d)
    c = cuda(d)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    loss, lse = ngr.fused_linear_cross_entropy(c["x"], c["W"], c["target"], stream=side)
    dx, dW = ngr.fused_linear_cross_entropy_backward(c["dloss"], lse, c["x"], c["W"], c["target"], stream=side)
    side.synchronize()
    assert torch.equal(loss, want["loss"]) and torch.equal(dx, want["dx"]) and torch.equal(dW, want["dW"])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        loss, lse = ngr.fused_linear_cross_entropy(c["x"], c["W"], c["target"])
        dx, dW = ngr.fused_linear_cross_entropy_backward(c["dloss"], lse, c["x"], c["W"], c["target"])
    # other inputs, another number of counted tokens
    e = R.case(270, 192, 1200, torch.bfloat16, seed=11, ignored=0.8)
    for k in c:
        c[k].copy_(e[k])
    graph.replay()
    torch.cuda.synchronize()
    val, tol = R.reference(e, 1.0, e["dloss"])
    for got, k in ((loss, "loss"), (lse, "lse"), (dx, "dx"), (dW, "dW")):
        R.check(got, val[k], tol[k], "replayed " + k)


def test_gradient_against_differences():
    """<gradient, direction> against the central difference of the float64
    forward along that direction."""
    d = R.case(20, 40, 90, torch.float16, seed=12, ignored=0.2)
    got = run(d)
    val, tol = R.reference(d, 1.0, d["dloss"])
    e = 1e-4
    g = torch.Generator("cpu")
    g.manual_seed(13)
    for k in ("x", "W"):
        t = torch.randn(d[k].shape, generator=g, dtype=torch.float64)
        side = []
        for sign in (1, -1):
            w = dict(d)
            w[k] = d[k].double() + sign * e * t
            z = w["x"].double() @ w["W"].double().T
            loss = torch.logsumexp(z, 1) - z.gather(1, d["target"].clamp(min=0)[:, None])[:, 0]
            side.append((torch.where(d["target"] >= 0, loss, 0.0) * d["dloss"].double()).sum())
        slope = ((side[0] - side[1]) / (2 * e)).item()
        mine = (got["d" + k].double().cpu() * t).sum().item()
        assert abs(mine - slope) <= (tol["d" + k] * t.abs()).sum().item() + 1e-6 * abs(slope), (k, mine, slope)
