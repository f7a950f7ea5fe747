"""The linear cross entropy's entry points on the host: refusals before
anything is launched, workspace sizes, the helper's own checks."""
import pytest
import torch

import normalization_gemm_row_gb300 as pkg
from normalization_gemm_row_gb300 import binding as B

A = 0x10000      # a fake address: never dereferenced
WS = A * 16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    pkg.build()


def forward(**kw):
    a = dict(x=A, W=A, t=A, scale=1.0, M=4, K=64, V=100, dtype=0, loss=A, lse=A, ws=WS, bytes=1 << 20)
    a.update(kw)
    return B.ngr_fused_linear_cross_entropy(a["x"], a["W"], a["t"], a["scale"], a["M"], a["K"], a["V"], a["dtype"],
                                            a["loss"], a["lse"], a["ws"], a["bytes"], None)


def backward(**kw):
    a = dict(g=A, gl=A, lse=A, x=A, W=A, t=A, scale=1.0, M=4, K=64, V=100, dtype=0, dx=A, dW=A, ws=WS, bytes=1 << 24)
    a.update(kw)
    return B.ngr_fused_linear_cross_entropy_backward(a["g"], a["gl"], a["lse"], a["x"], a["W"], a["t"], a["scale"], a["M"],
                                                     a["K"], a["V"], a["dtype"], a["dx"], a["dW"], a["ws"], a["bytes"], None)


COMMON = [(dict(M=-1), -2), (dict(K=0), -2), (dict(V=0), -2), (dict(V=1 << 31), -2), (dict(dtype=7), -4),
          (dict(x=None), -1), (dict(W=None), -1), (dict(t=None), -1), (dict(scale=float("nan")), -9),
          (dict(scale=float("inf")), -9), (dict(x=A + 1), -3), (dict(W=A + 8), -3), (dict(K=60, W=A + 1), -3),
          (dict(t=A + 4), -3), (dict(ws=None), -5), (dict(bytes=512), -5), (dict(ws=WS + 128), -3)]


@pytest.mark.parametrize("kw,expect", COMMON + [
    (dict(loss=None), -1), (dict(lse=None), -1), (dict(loss=A + 2), -3), (dict(M=0), 0), (dict(M=0, ws=None), 0)])
def test_forward_refuses(kw, expect):
    assert forward(**kw) == expect


@pytest.mark.parametrize("kw,expect", COMMON + [
    (dict(dx=None, dW=None), -1), (dict(g=None, gl=None), -1), (dict(lse=None), -1), (dict(dx=A + 1), -3),
    (dict(dW=A + 1), -3), (dict(g=A + 2), -3), (dict(M=0, dW=None), 0)])
def test_backward_refuses(kw, expect):
    assert backward(**kw) == expect


def test_workspace_bytes():
    f = B.ngr_linear_cross_entropy_workspace_bytes
    a256 = lambda v: (v + 255) // 256 * 256
    M, K, V = 1000, 512, 50000
    common = 256 + 256 + 2 * a256(4 * M) + 1024 * K * 2
    # two (maximum, sum) pairs a token for each tile of 128 to 256 entries
    assert f(0, M, K, V) in [common + a256(2 * -(-V // w) * M * 8) + a256(4 * M) for w in range(128, 257, 32)]
    # ragged width: W's padded copy
    assert f(0, M, K - 1, V) == f(0, M, K, V) + a256(V * K * 2)
    # backward: never more than 256 MB of dz (or 4096 entries), whatever the vocabulary
    assert f(1, 8192, 4096, 1 << 20) - f(1, 8192, 4096, 1 << 18) == 0
    assert f(1, 8192, 4096, 131072) < (256 << 20) + 8192 * 4096 * (2 + 4) + (1 << 20)
    # the logits of 8192 x 131072 in 16 bits alone would take 2 GB
    for bad in ((0, -1, 8, 8), (1, 1, 0, 8), (1, 1, 8, 0)):
        assert f(*bad) == 0


def test_helper_refuses():
    x, W = torch.zeros(4, 8, dtype=torch.float16), torch.zeros(10, 8, dtype=torch.float16)
    t = torch.zeros(4, dtype=torch.int64)
    with pytest.raises(ValueError, match="CUDA"):
        pkg.fused_linear_cross_entropy(x, W, t)
    with pytest.raises(ValueError, match="V, K"):
        pkg.fused_linear_cross_entropy(x, W[:, :4], t)
    with pytest.raises(TypeError, match="int64"):
        pkg.fused_linear_cross_entropy(x, W, t.int())
    with pytest.raises(ValueError, match="one entry"):
        pkg.fused_linear_cross_entropy(x, W, t[:3])
