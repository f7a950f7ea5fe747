"""The linear cross entropy where offsets pass 31 bits: a weight of 2.2e9
elements, and as many of hidden states.  Tolerances: those of
ce_reference.py, on the entries that are looked at."""
import pytest
import torch

import normalization_gemm_row_gb300 as ngr
import ce_reference as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    ngr.build()
    torch.cuda.init()


@pytest.mark.parametrize("K", [8192, 8191])
def test_large_weight(K):
    M, V = 3, 270000
    W = torch.empty((V, K), dtype=torch.bfloat16, device="cuda").normal_(0.0, K ** -0.5)
    target = torch.tensor([0, V // 2, V - 1], device="cuda")
    x = (torch.randn((M, K), device="cuda") + 6.0 * W[target].float()).bfloat16()
    g = torch.tensor([0.5, 1.0, 0.25], device="cuda")
    loss, lse = ngr.fused_linear_cross_entropy(x, W, target)
    dx, dW = ngr.fused_linear_cross_entropy_backward(g, lse, x, W, target)
    X = x.double()
    z = torch.cat([X @ W[v:v + 30000].double().T for v in range(0, V, 30000)], 1)
    top = torch.logsumexp(z, 1)
    # (a logit's error as ce_reference.py has it, its terms' sizes by Cauchy and Schwarz)
    ez = (K / 16 + 16) * 2.0 ** -23 * X.norm(dim=1) * 1.25
    el = ez + 80 * 2.0 ** -23 + 2.0 ** -22 * top.abs()
    assert ((lse.double() - top).abs() <= el).all()
    assert ((loss.double() - (top - z[torch.arange(M), target])).abs() <= el + ez + 2.0 ** -22 * top.abs()).all()
    p = torch.exp(z - top[:, None])
    p[torch.arange(M), target] -= 1.0
    dz = g.double()[:, None] * p
    edz = g.double()[:, None] * torch.exp(z - top[:, None]) * (ez + el + 2.0 ** -20)[:, None] + 1.01 * 2.0 ** -8 * dz.abs()
    for v in (0, V // 2 - 64, V - 128):
        want = dz[:, v:v + 128].T @ X
        size = edz[:, v:v + 128].T @ X.abs() + 100 * 2.0 ** -23 * (dz[:, v:v + 128].abs().T @ X.abs())
        assert ((dW[v:v + 128].double() - want).abs() <= size + 2.0 ** -8 * want.abs() + 1e-38).all(), v
    want, size = 0.0, 0.0
    for v in range(0, V, 30000):
        w = W[v:v + 30000].double()
        want = want + dz[:, v:v + 30000] @ w
        size = size + (edz[:, v:v + 30000] + (V / 16 + 80) * 2.0 ** -23 * dz[:, v:v + 30000].abs()) @ w.abs()
    assert ((dx.double() - want).abs() <= size + 2.0 ** -8 * want.abs() + 1e-38).all()


def test_many_tokens():
    M, K, V, tail = 270000, 8192, 300, 64
    d = R.case(tail, K, V, torch.bfloat16, seed=1, ignored=0.3)
    x = torch.empty((M, K), dtype=torch.bfloat16, device="cuda").normal_()
    target = torch.randint(0, V, (M,), device="cuda")
    target[::3] = -1
    dloss = torch.rand(M, device="cuda") * 0.1 + 0.01
    x[M - tail:], target[M - tail:], dloss[M - tail:] = d["x"].cuda(), d["target"].cuda(), d["dloss"].cuda()
    W = d["W"].cuda()
    loss, lse = ngr.fused_linear_cross_entropy(x, W, target)
    dx, _ = ngr.fused_linear_cross_entropy_backward(dloss, lse, x, W, target, need_dW=False)
    val, tol = R.reference(d, 1.0, d["dloss"])
    for got, k in ((loss, "loss"), (lse, "lse"), (dx, "dx")):
        R.check(got[M - tail:], val[k], tol[k], k)
    off = target < 0
    assert (dx[off] == 0).all() and (loss[off] == 0).all() and (loss[~off] > 0).all()
