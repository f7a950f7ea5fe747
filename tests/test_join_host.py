"""The block join's entry points on the host: refusals before anything is
launched, workspace sizes, the helper's own checks."""
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
    a = dict(norm1=2, norm2=2, x=A, residual=A, gate=A, rpg=4, gamma1=A, beta1=A, gamma2=A, beta2=A, eps1=1e-5, eps2=1e-5,
             rs=1.0, bs=1.0, M=4, N=64, dtype=0, h=A, y=A, stats=A)
    a.update(kw)
    return B.ngr_fused_norm_gate_residual_norm(
        a["norm1"], a["norm2"], a["x"], a["residual"], a["gate"], a["rpg"], a["gamma1"], a["beta1"], a["gamma2"], a["beta2"],
        a["eps1"], a["eps2"], a["rs"], a["bs"], a["M"], a["N"], a["dtype"], a["h"], a["y"], a["stats"], None)


def backward(**kw):
    a = dict(norm1=2, norm2=2, dy=A, dh=A, x=A, residual=A, gate=A, rpg=4, gamma1=A, beta1=A, gamma2=A, beta2=A, stats=A,
             rs=1.0, bs=1.0, M=4, N=64, dtype=0, dx=A, dr=A, dg=A, v=A, ws=WS, bytes=1 << 20)
    a.update(kw)
    return B.ngr_fused_norm_gate_residual_norm_backward(
        a["norm1"], a["norm2"], a["dy"], a["dh"], a["x"], a["residual"], a["gate"], a["rpg"], a["gamma1"], a["beta1"],
        a["gamma2"], a["stats"], a["rs"], a["bs"], a["M"], a["N"], a["dtype"], a["dx"], a["dr"], a["dg"], a["v"],
        a["v"], a["v"], a["v"], a["ws"], a["bytes"], None)


@pytest.mark.parametrize("kw,expect", [
    (dict(norm1=3), -9), (dict(norm2=-1), -9), (dict(rpg=0), -9), (dict(rpg=-5), -9), (dict(eps1=-1.0), -9),
    (dict(eps2=float("nan")), -9), (dict(rs=float("inf")), -9), (dict(bs=float("nan")), -9),
    (dict(gamma1=None), -1), (dict(norm1=1, beta1=None), -1), (dict(gamma2=None), -1), (dict(norm2=1, beta2=None), -1),
    (dict(x=None), -1), (dict(h=None), -1), (dict(y=None), -1),
    (dict(M=-1), -2), (dict(N=0), -2), (dict(N=65537), -2), (dict(M=1 << 31), -2), (dict(dtype=2), -4),
    (dict(x=A + 1), -3), (dict(residual=A + 1), -3), (dict(gate=A + 1), -3), (dict(y=A + 1), -3), (dict(stats=A + 8), -3),
    (dict(M=0), 0), (dict(M=0, x=None), 0)])
def test_forward_refuses(kw, expect):
    assert forward(**kw) == expect


@pytest.mark.parametrize("kw,expect", [
    (dict(norm1=5), -9), (dict(rpg=0), -9), (dict(gamma1=None), -1), (dict(norm2=1, gamma2=None), -1),
    (dict(x=None), -1), (dict(stats=None), -1), (dict(dx=None), -1), (dict(dy=None, dh=None), -1),
    (dict(norm2=0, dh=None), -1), (dict(residual=None), -1), (dict(N=70000), -2), (dict(dtype=-1), -4),
    (dict(dy=A + 1), -3), (dict(dg=A + 1), -3), (dict(v=A + 1), -3), (dict(stats=A + 4), -3),
    (dict(ws=None), -5), (dict(bytes=256), -5), (dict(ws=WS + 16), -3)])
def test_backward_refuses(kw, expect):
    assert backward(**kw) == expect


def test_workspace_bytes():
    f = B.ngr_norm_gate_residual_norm_workspace_bytes
    # a row of FP32 sums for each CTA (two an SM at this width) and sum
    assert f(2, 2, 0, 8192, 4096) == 256 + 2 * 304 * 4096 * 4
    assert f(2, 2, 8192, 8192, 4096) == f(2, 2, 0, 8192, 4096)
    assert f(0, 0, 0, 100, 64) == 256                         # no sums without a norm or a gate
    assert f(0, 2, 1, 400, 4096) == 256 + 304 * 4096 * 4      # dgate of one token each: written directly
    for bad in ((3, 2, 0, 8, 8), (2, 2, 0, -1, 8), (2, 2, 0, 8, 0), (2, 2, 0, 8, 65537)):
        assert f(*bad) == 0
    assert f(2, 2, 0, 0, 64) == 256
    # a few rows of sums per CTA, or one per gate row of 16 tokens or more
    for M in (1, 17, 1000, 100000):
        for g in (0, 1, 7, M):
            for N in (8, 999, 16384, 65536):
                assert f(1, 1, g, M, N) <= 256 + (2 * 4 * 1520 + 2 * 1520 + 2 * M) * N * 4


def test_helper_refuses():
    t = torch.zeros(4, 8, dtype=torch.float16)
    with pytest.raises(ValueError, match="CUDA"):
        pkg.fused_norm_gate_residual_norm(t, t, gamma1=t[0], gamma2=t[0])
    with pytest.raises(ValueError, match="residual"):
        pkg.fused_norm_gate_residual_norm(t, t[:2], gamma1=t[0], gamma2=t[0])
    with pytest.raises(ValueError, match="gate"):
        pkg.fused_norm_gate_residual_norm(t, t, gate=t[:3], gamma1=t[0], gamma2=t[0])
    with pytest.raises(ValueError, match="column"):
        pkg.fused_norm_gate_residual_norm(t, t, gamma1=t[0, :4], gamma2=t[0])
