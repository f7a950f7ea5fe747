"""GPU parity of the block join (norm, gate, residual, norm) and its gradient
against the formulas in float64, at the sizes, gates and addresses where the
kernels change path.  The tolerance is derived in join_reference.py."""
import pytest
import torch

import normalization_gemm_row_gb300 as ngr
from normalization_gemm_row_gb300 import binding as B
import join_reference as R

pytestmark = pytest.mark.gpu
NONE, LAYER, RMS = 0, 1, 2
DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _built():
    ngr.build()
    torch.cuda.init()


def cuda(d):
    return {k: (v.cuda() if v is not None else None) for k, v in d.items()}


def how(c, norm1, norm2, eps=1e-5, a=1.0, s=1.0):
    return dict(gate=c["gate"], norm1=norm1, gamma1=c["gamma1"], beta1=c["beta1"], eps1=eps, norm2=norm2,
                gamma2=c["gamma2"], beta2=c["beta2"], eps2=eps, residual_scale=a, block_scale=s)


def run(d, norm1, norm2, **kw):
    c = cuda(d)
    args = how(c, norm1, norm2, **kw)
    h, y, st = ngr.fused_norm_gate_residual_norm(c["x"], c["residual"], return_stats=True, **args)
    got = {"h": h, "y": y}
    got.update(ngr.fused_norm_gate_residual_norm_backward(c["dy"], c["dh"], c["x"], c["residual"], st, **args))
    return got, st


def compare(d, norm1, norm2, what, **kw):
    got, st = run(d, norm1, norm2, **kw)
    val, mag = R.reference(d, norm1, norm2, **kw)
    for k, v in val.items():
        if v is None:
            assert got[k] is None
        else:
            R.check(got[k], v, mag[k], d["x"].dtype, f"{what} {k}")
    for k, v in got.items():
        assert v is None or k in val, k
    return got, st


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("gates", [0, 1, 3, 6])
@pytest.mark.parametrize("norm2", [NONE, LAYER, RMS])
@pytest.mark.parametrize("norm1", [NONE, LAYER, RMS])
def test_every_form(norm1, norm2, gates, dtype):
    for M, N in ((6, 264), (6, 131)):
        d = R.case(M, N, norm1, norm2, gates, DTYPES[dtype], seed=norm1 * 9 + norm2 * 3 + gates)
        compare(d, norm1, norm2, f"{M}x{N}", a=1.25, s=0.5)


# Around the changes of path: one warp a row, several, two and four vectors a
# thread, clusters (N above 16384; above 10240 with five sums), single
# elements, single rows, more rows than CTAs.
SHAPES = [(1, 1), (2, 7), (1, 8), (5, 33), (700, 8), (31, 256), (9, 257), (4, 1152), (3, 2048), (2, 2056), (3, 4095),
          (2, 4104), (5, 8192), (2, 8200), (1, 10248), (2, 14337), (2, 16384), (3, 16392), (2, 16411), (2, 40000),
          (1, 65536), (305, 520)]


@pytest.mark.parametrize("M,N", SHAPES)
def test_sizes(M, N):
    for norm1, norm2, gates, dtype in ((LAYER, LAYER, 1, torch.float16), (RMS, RMS, 1, torch.bfloat16),
                                       (NONE, RMS, 0, torch.bfloat16)):
        d = R.case(M, N, norm1, norm2, gates, dtype, seed=M + N)
        compare(d, norm1, norm2, f"{M}x{N} {norm1}{norm2}")


@pytest.mark.parametrize("M,gates", [(1000, 8), (1000, 200), (400, 400), (320, 160), (2000, 2)])
def test_gate_groups(M, gates):
    """Fewer groups than CTAs, more, as many as rows: dgate from partial
    sums and directly."""
    d = R.case(M, 72, LAYER, RMS, gates, torch.bfloat16, seed=M + gates)
    compare(d, LAYER, RMS, f"{M} rows, {gates} gates")


@pytest.mark.parametrize("M,N,gates", [(640, 4900, 16), (160, 8200, 10), (300, 10252, 1)])
def test_last_sums_by_four_columns(M, N, gates):
    for norm1, dtype in ((LAYER, torch.float16), (NONE, torch.bfloat16)):
        d = R.case(M, N, norm1, LAYER, gates, dtype, seed=M + N)
        compare(d, norm1, LAYER, f"{M}x{N}, {gates} gates", s=1.5)


@pytest.mark.parametrize("M,N,gates", [(1400, 1001, 1), (4000, 131, 2), (1300, 2050, 0), (2403, 517, 3), (1801, 36, 1),
                                       (900, 5003, 1), (700, 20004, 0)])
def test_many_rows_that_are_not_aligned(M, N, gates):
    """The gradient's CTAs take every 8th, 4th or 2nd row: rows that start
    alike."""
    for norm1, norm2, dtype in ((LAYER, LAYER, torch.float16), (RMS, RMS, torch.bfloat16)):
        d = R.case(M, N, norm1, norm2, gates, dtype, seed=M + N)
        compare(d, norm1, norm2, f"{M}x{N}", a=0.75)


def test_ragged_last_group():
    """M need not be a multiple of rows_per_gate at the C entry."""
    M, N, rpg = 10, 40, 4
    d = R.case(M, N, RMS, RMS, 3, torch.float16, seed=5)
    c = cuda(d)
    h, y = torch.empty_like(c["x"]), torch.empty_like(c["x"])
    st = torch.empty((M, 4), device="cuda")
    s = torch.cuda.current_stream().cuda_stream
    p = lambda t: None if t is None else t.data_ptr()
    assert B.ngr_fused_norm_gate_residual_norm(RMS, RMS, p(c["x"]), p(c["residual"]), p(c["gate"]), rpg, p(c["gamma1"]), None,
                                               p(c["gamma2"]), None, 1e-5, 1e-5, 1.0, 1.0, M, N, 0, p(h), p(y), p(st), s) == 0
    n = B.ngr_norm_gate_residual_norm_workspace_bytes(RMS, RMS, rpg, M, N)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    dx, dr, dg = torch.empty_like(h), torch.empty_like(h), torch.empty_like(c["gate"])
    assert B.ngr_fused_norm_gate_residual_norm_backward(
        RMS, RMS, p(c["dy"]), p(c["dh"]), p(c["x"]), p(c["residual"]), p(c["gate"]), rpg, p(c["gamma1"]), None, p(c["gamma2"]),
        p(st), 1.0, 1.0, M, N, 0, p(dx), p(dr), p(dg), None, None, None, None, p(ws), n, s) == 0
    assert B.ngr_workspace_error(p(ws), s) == 0
    # the same rows with two rows of zeros behind them
    big = {k: (torch.cat([v, torch.zeros(2, N, dtype=v.dtype)]) if k in ("x", "residual", "dy", "dh") else v) for k, v in d.items()}
    val, mag = R.reference(big, RMS, RMS)
    for got, k in ((h, "h"), (y, "y"), (dx, "dx"), (dr, "dresidual")):
        R.check(got, val[k][:M], mag[k][:M], torch.float16, k)
    R.check(dg, val["dgate"], mag["dgate"], torch.float16, "dgate")


@pytest.mark.parametrize("dtype", list(DTYPES))
def test_hard_rows(dtype):
    """Rows far from zero mean, constant rows, zero rows, rows with one very
    large channel."""
    d = R.case(8, 4096, LAYER, LAYER, 1, DTYPES[dtype], seed=3)
    for k in ("x", "residual"):
        d[k][0] = 2.5
        d[k][1] = 0.0
        d[k][2] = (1000 + torch.arange(4096) % 7).to(DTYPES[dtype])
        d[k][3, 17] = 20000.0
    for norm1, norm2 in ((LAYER, LAYER), (RMS, RMS), (NONE, LAYER)):
        e = dict(d)
        if norm1 != LAYER:
            e["beta1"] = None
        if norm2 != LAYER:
            e["beta2"] = None
        if norm1 == NONE:
            e["gamma1"] = None
        c = cuda(e)
        h, y = ngr.fused_norm_gate_residual_norm(c["x"], c["residual"], **how(c, norm1, norm2, eps=1e-3))
        val, mag = R.reference(e, norm1, norm2, eps=1e-3)
        R.check(h, val["h"], mag["h"], DTYPES[dtype], "h")
        R.check(y, val["y"], mag["y"], DTYPES[dtype], "y")


def test_no_residual_and_missing_gradients():
    d = R.case(7, 320, RMS, LAYER, 1, torch.bfloat16, seed=11, residual=False)
    got, _ = compare(d, RMS, LAYER, "no residual")
    assert got["dresidual"] is None
    for gone in ("dy", "dh"):
        e = R.case(7, 320, RMS, LAYER, 1, torch.bfloat16, seed=12)
        e[gone] = None
        compare(e, RMS, LAYER, f"no {gone}")


@pytest.mark.parametrize("N", [264, 261])
def test_any_even_address(N):
    """Rows that start one element off a 16-byte boundary."""
    d = R.case(9, N, LAYER, RMS, 3, torch.float16, seed=N)
    c = cuda(d)

    def off(t):
        if t is None:
            return None
        return torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")[1:].view(t.shape).copy_(t)

    c = {k: off(v) for k, v in c.items()}
    args = how(c, LAYER, RMS)
    h, y, st = ngr.fused_norm_gate_residual_norm(c["x"], c["residual"], return_stats=True, h=off(torch.zeros_like(c["x"])),
                                                 out=off(torch.zeros_like(c["x"])), **args)
    got = {"h": h, "y": y}
    got.update(ngr.fused_norm_gate_residual_norm_backward(c["dy"], c["dh"], c["x"], c["residual"], st, **args))
    val, mag = R.reference(d, LAYER, RMS)
    for k, v in val.items():
        if v is not None:
            R.check(got[k], v, mag[k], torch.float16, k)


def test_outputs_in_place_and_nothing_else_written():
    d = R.case(5, 512, RMS, RMS, 1, torch.bfloat16, seed=2)
    c = cuda(d)
    want = ngr.fused_norm_gate_residual_norm(c["x"], c["residual"], **how(c, RMS, RMS))
    pad = torch.full((7, 512), 3.0, dtype=torch.bfloat16, device="cuda")
    pad2 = pad.clone()
    pad[:5], pad2[:5] = c["x"], c["residual"]
    h, y = ngr.fused_norm_gate_residual_norm(pad[:5], pad2[:5], h=pad2[:5], out=pad[:5], **how(c, RMS, RMS))
    assert h.data_ptr() == pad2.data_ptr() and y.data_ptr() == pad.data_ptr()
    assert torch.equal(h, want[0]) and torch.equal(y, want[1])
    assert (pad[5:] == 3).all() and (pad2[5:] == 3).all()


def test_same_call_same_bits():
    d = R.case(1000, 1152, LAYER, LAYER, 8, torch.bfloat16, seed=4)
    a, sa = run(d, LAYER, LAYER)
    b, sb = run(d, LAYER, LAYER)
    assert torch.equal(sa, sb)
    for k in a:
        assert torch.equal(a[k], b[k]), k


def test_empty_batch():
    c = cuda(R.case(0, 64, LAYER, LAYER, 0, torch.float16, seed=1))
    args = how(c, LAYER, LAYER)
    h, y, st = ngr.fused_norm_gate_residual_norm(c["x"], c["residual"], return_stats=True, **args)
    g = ngr.fused_norm_gate_residual_norm_backward(c["dy"], c["dh"], c["x"], c["residual"], st, **args)
    assert h.shape == (0, 64) and g["dx"].shape == (0, 64)
    for k in ("dgamma1", "dbeta1", "dgamma2", "dbeta2"):
        assert (g[k] == 0).all(), k


def test_captured_and_on_another_stream():
    d = R.case(40, 2048, RMS, RMS, 1, torch.bfloat16, seed=8)
    c = cuda(d)
    args = how(c, RMS, RMS)
    want, _ = run(d, RMS, RMS)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    h, y, st = ngr.fused_norm_gate_residual_norm(c["x"], c["residual"], return_stats=True, stream=side, **args)
    g = ngr.fused_norm_gate_residual_norm_backward(c["dy"], c["dh"], c["x"], c["residual"], st, stream=side, **args)
    side.synchronize()
    assert torch.equal(h, want["h"]) and torch.equal(g["dx"], want["dx"]) and torch.equal(g["dgamma2"], want["dgamma2"])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        h, y, st = ngr.fused_norm_gate_residual_norm(c["x"], c["residual"], return_stats=True, **args)
        g = ngr.fused_norm_gate_residual_norm_backward(c["dy"], c["dh"], c["x"], c["residual"], st, **args)
    c["x"].mul_(0.5)
    c["dy"].mul_(2.0)
    graph.replay()
    torch.cuda.synchronize()
    e = {k: (v.cpu() if v is not None else None) for k, v in c.items()}
    val, mag = R.reference(e, RMS, RMS)
    for got, k in ((h, "h"), (y, "y"), (g["dx"], "dx"), (g["dgamma1"], "dgamma1"), (g["dgate"], "dgate")):
        R.check(got, val[k], mag[k], torch.bfloat16, "replayed " + k)


@pytest.mark.parametrize("norm1,norm2", [(LAYER, RMS), (RMS, LAYER)])
def test_gradient_against_differences(norm1, norm2):
    """<gradient, direction> against the central difference of the float64
    forward along that direction (step e: its error is of order e^2 times
    the third derivative, below the rounding of the gradients here)."""
    d = R.case(12, 96, norm1, norm2, 3, torch.float16, seed=21)
    got, _ = run(d, norm1, norm2)
    val, mag = R.reference(d, norm1, norm2)
    g = torch.Generator("cpu")
    g.manual_seed(22)
    names = [k for k in ("x", "residual", "gate", "gamma1", "beta1", "gamma2", "beta2") if d[k] is not None]
    e = 1e-4
    for k in names:
        t = torch.randn(d[k].shape, generator=g, dtype=torch.float64)
        sides = []
        for sign in (1, -1):
            w = {n: (v.double() if v is not None else None) for n, v in d.items()}
            w[k] = w[k] + sign * e * t
            h, y = R.forward(w, norm1, norm2)
            sides.append((h * w["dh"]).sum() + (y * w["dy"]).sum())
        slope = ((sides[0] - sides[1]) / (2 * e)).item()
        mine = (got["d" + k].double().cpu() * t).sum().item()
        tol = ((R.U[torch.float16] * val["d" + k].abs() + R.SLACK * mag["d" + k]) * t.abs()).sum().item()
        assert abs(mine - slope) <= tol + 1e-5 * abs(slope), (k, mine, slope, tol)


def test_statistics():
    d = R.case(6, 777, LAYER, RMS, 0, torch.bfloat16, seed=6, mean=5.0)
    _, st = run(d, LAYER, RMS)
    x = d["x"].double()
    h, _ = R.forward({k: (v.double() if v is not None else None) for k, v in d.items()}, LAYER, RMS)
    want = torch.stack([x.mean(1), 1 / torch.sqrt(x.var(1, unbiased=False) + 1e-5), torch.zeros(6, dtype=torch.float64),
                        1 / torch.sqrt((h * h).mean(1) + 1e-5)], 1)
    assert ((st.double().cpu() - want).abs() <= 2.0 ** -18 * want.abs() + 1e-12).all()
