"""The block join where its kernels take other paths than at ordinary sizes:
arrays that start at different places, few tokens to a gate row in wide and
unaligned rows, infinities and NaN, long columns of sums, and offsets past 31
bits.  Tolerances from join_reference.py but where one is derived here."""
import pytest
import torch

import normalization_gemm_row_gb300 as ngr
import join_reference as R
import test_join_gpu as J

pytestmark = pytest.mark.gpu
NONE, LAYER, RMS = J.NONE, J.LAYER, J.RMS


@pytest.fixture(scope="module", autouse=True)
def _built():
    ngr.build()
    torch.cuda.init()


def at(t, off):
    """t (or room for its like) `off` elements behind a 16-byte boundary."""
    return torch.empty(t.numel() + 8, dtype=t.dtype, device="cuda")[off:off + t.numel()].view(t.shape).copy_(t)


@pytest.mark.parametrize("N", [3, 40, 999, 1000, 1025, 4104, 8192, 8200, 16384, 16385, 20003, 40000])
def test_arrays_that_start_at_different_places(N):
    """One element at a time, forward and backward, in one warp, several and
    clusters."""
    for norm1, norm2, gates, dtype in ((LAYER, LAYER, 0, torch.float16), (RMS, RMS, 5, torch.bfloat16),
                                       (NONE, RMS, 1, torch.bfloat16), (LAYER, LAYER, 5, torch.bfloat16)):
        d = R.case(5, N, norm1, norm2, gates, dtype, seed=N + gates)
        c = J.cuda(d)
        for i, k in enumerate(("x", "residual", "dy", "dh")):
            c[k] = at(c[k], 1 + 2 * i)
        for i, k in enumerate(("gate", "gamma1", "beta1", "gamma2", "beta2")):
            if c[k] is not None:
                c[k] = at(c[k], i)
        args = J.how(c, norm1, norm2, a=0.75)
        h, y, st = ngr.fused_norm_gate_residual_norm(c["x"], c["residual"], return_stats=True, h=at(c["x"], 4),
                                                     out=at(c["x"], 2), **args)
        got = {"h": h, "y": y}
        got.update(ngr.fused_norm_gate_residual_norm_backward(c["dy"], c["dh"], c["x"], c["residual"], st, **args))
        val, mag = R.reference(d, norm1, norm2, a=0.75)
        for k, v in val.items():
            if v is not None:
                R.check(got[k], v, mag[k], dtype, f"5x{N} {norm1}{norm2} {k}")


@pytest.mark.parametrize("N", [257, 2048, 2056, 4099, 5003, 7680, 7688, 8200, 16392, 20001])
@pytest.mark.parametrize("tokens", [1, 3, 15])
def test_few_tokens_to_a_gate_row(N, tokens):
    gates = 4 if N > 6000 else 9
    for norm1, norm2, dtype in ((LAYER, LAYER, torch.bfloat16), (RMS, RMS, torch.float16)):
        d = R.case(gates * tokens, N, norm1, norm2, gates, dtype, seed=N + tokens)
        J.compare(d, norm1, norm2, f"{gates} gates of {tokens} tokens x {N}", s=1.25)


@pytest.mark.parametrize("M,N,gates", [(2100, 264, 2100), (1400, 1157, 700), (930, 2048, 310)])
def test_more_gate_rows_than_ctas(M, N, gates):
    for norm1, norm2 in ((LAYER, LAYER), (RMS, NONE), (NONE, RMS)):
        d = R.case(M, N, norm1, norm2, gates, torch.bfloat16, seed=M)
        J.compare(d, norm1, norm2, f"{M}x{N}, {gates} gates")


@pytest.mark.parametrize("N", [72, 75, 2048, 4099])
@pytest.mark.parametrize("norm", [LAYER, RMS])
def test_rows_that_are_not_finite(norm, N):
    """Infinities and NaN stay in their row (at its ends too, where unaligned
    rows share a 16-byte word) and, in sums, in their gate row's group."""
    M, bad = 12, {1: float("inf"), 4: float("nan"), 7: float("-inf"), 11: float("nan")}
    d = R.case(M, N, norm, norm, 4, torch.float16, seed=N + norm)
    plain, _ = J.run(d, norm, norm)
    for k in ("x", "residual", "dy", "dh"):
        e = dict(d)
        e[k] = d[k].clone()
        for i, (row, v) in enumerate(bad.items()):
            e[k][row, (0, N - 1, N // 2, 0)[i]] = v
        got, _ = J.run(e, norm, norm)
        good = torch.tensor([i not in bad for i in range(M)])
        for o in ("h", "y", "dx", "dresidual"):
            assert torch.equal(got[o].cpu()[good], plain[o].cpu()[good]), (k, o)
        h, y = R.forward({n: (v.double() if v is not None else None) for n, v in e.items()}, norm, norm)
        for o, v in (("h", h), ("y", y)):
            a = got[o].double().cpu()
            assert torch.equal(torch.isnan(a), torch.isnan(v)) and torch.equal(torch.isinf(a), torch.isinf(v)), (k, o)
    e = dict(d)
    e["dh"] = d["dh"].clone()
    e["dh"][4] = float("nan")
    got, _ = J.run(e, norm, norm)
    clean = torch.tensor([True, False, True, True])
    assert torch.equal(got["dgate"].cpu()[clean], plain["dgate"].cpu()[clean])
    assert torch.isnan(got["dgate"][1]).all() and torch.isnan(got["dgamma1"]).all()
    assert torch.equal(got["dgamma2"], plain["dgamma2"])


@pytest.mark.parametrize("M,N,gates,dtype", [(400000, 40, 1, torch.float16), (60000, 1157, 3, torch.bfloat16),
                                             (40000, 4096, 0, torch.float16)])
def test_long_columns(M, N, gates, dtype):
    """Many rows to a CTA, whose column sums are chains of additions: M / 152
    of them at most (a row is one CTA's at these widths, and every SM has one),
    an additional half step of FP32 each beside the terms' own."""
    d = J.cuda(R.case(16 * max(1, gates), N, LAYER, LAYER, gates, dtype, seed=N))
    g = torch.Generator("cuda")
    g.manual_seed(M)
    for k, mean in (("x", 0.3), ("residual", 0.0), ("dy", 0.5), ("dh", -0.25)):
        d[k] = torch.empty((M, N), dtype=dtype, device="cuda").normal_(mean, 1.0, generator=g)
    args = J.how(d, LAYER, LAYER)
    h, y, st = ngr.fused_norm_gate_residual_norm(d["x"], d["residual"], return_stats=True, **args)
    got = ngr.fused_norm_gate_residual_norm_backward(d["dy"], d["dh"], d["x"], d["residual"], st, **args)
    slack = (128 + M / 152) * 2.0 ** -24
    val = {k: 0.0 for k in ("dgamma1", "dbeta1", "dgamma2", "dbeta2")}
    mag = dict(val)
    rows_per_gate = M // max(1, gates)
    val["dgate"], mag["dgate"] = [torch.zeros((max(1, gates), N), dtype=torch.float64, device="cuda") for _ in range(2)]
    g1, b1, g2 = (d[k].double() for k in ("gamma1", "beta1", "gamma2"))
    for r in range(0, M, 20000):
        x, res, dy, dh = (d[k][r:r + 20000].double() for k in ("x", "residual", "dy", "dh"))
        group = torch.arange(r, r + x.shape[0], device="cuda") // rows_per_gate
        gate = d["gate"].double()[group] if gates else torch.ones((1, 1), dtype=torch.float64, device="cuda")
        c = x - x.mean(1, keepdim=True)
        u1 = c / torch.sqrt((c * c).mean(1, keepdim=True) + 1e-5)
        n = g1 * u1 + b1
        hh = res + gate * n
        c = hh - hh.mean(1, keepdim=True)
        root = torch.sqrt((c * c).mean(1, keepdim=True) + 1e-5)
        u2 = c / root
        q = g2 * dy
        D = dh + (q - q.mean(1, keepdim=True) - u2 * (q * u2).mean(1, keepdim=True)) / root
        # (the terms' sizes before anything cancels)
        big = dh.abs() + (q.abs() + q.abs().mean(1, keepdim=True) + u2.abs() * (q * u2).abs().mean(1, keepdim=True)) / root
        size1, size2 = u1.abs() + x.abs(), u2.abs() + hh.abs() / root
        for k, t, s in (("dgamma1", gate * D * u1, gate.abs() * big * size1), ("dbeta1", gate * D, gate.abs() * big),
                        ("dgamma2", dy * u2, dy.abs() * size2), ("dbeta2", dy, dy.abs())):
            val[k] = val[k] + t.sum(0)
            mag[k] = mag[k] + s.sum(0)
        for i in range(gates):
            mine = (group == i).double()[:, None]
            val["dgate"][i] += (mine * D * n).sum(0)
            mag["dgate"][i] += (mine * big * (g1.abs() * size1 + b1.abs())).sum(0)
    for k in val:
        if k == "dgate" and not gates:
            continue
        err = (got[k].double() - val[k]).abs()
        tol = R.U[dtype] * val[k].abs() + (1 + R.U[dtype]) * slack * mag[k] + R.TINY[dtype]
        big = torch.isinf(got[k].double()) & (val[k].abs() > torch.finfo(dtype).max * (1 - R.U[dtype]))
        assert ((err <= tol) | big).all(), (k, (err / tol)[~big].max().item())


@pytest.mark.parametrize("N", [8192, 8191])
def test_offsets_past_31_bits(N):
    """2.2e9 elements an array: the last rows are those of a short call."""
    M, tail = 270000, 96
    kw = dict(norm1=RMS, norm2=RMS, gamma1=torch.rand(N, device="cuda").bfloat16(), gamma2=torch.rand(N, device="cuda").bfloat16())
    big = [torch.empty((M, N), dtype=torch.bfloat16, device="cuda").normal_() for _ in range(4)]
    x, r, dy, dh = big
    h, y, st = ngr.fused_norm_gate_residual_norm(x, r, return_stats=True, **kw)
    # (rows whose 16-byte shifts are those of the first rows of an array)
    short = [t[M - tail:].clone() for t in big]
    hs, ys, ss = ngr.fused_norm_gate_residual_norm(short[0], short[1], return_stats=True, **kw)
    for a, b in ((h, hs), (y, ys), (st, ss)):
        assert torch.equal(a[M - tail:], b)
    del h, y
    g = ngr.fused_norm_gate_residual_norm_backward(dy, dh, x, r, st, **kw)
    s = ngr.fused_norm_gate_residual_norm_backward(short[2], short[3], short[0], short[1], ss, **kw)
    for k in ("dx", "dresidual"):
        assert torch.equal(g[k][M - tail:], s[k])
    for k in ("dgamma1", "dgamma2"):
        assert torch.isfinite(g[k]).all()
