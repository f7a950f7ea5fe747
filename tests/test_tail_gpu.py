"""A model's tail as it is used: two joins in a row, the head's cross entropy
on the second one's output, and the gradients back through all of them.

Each call is held to its formula in float64 on the inputs it was given (its
predecessors' outputs as stored), with the tolerances of join_reference.py and
ce_reference.py."""
import pytest
import torch

import normalization_gemm_row_gb300 as ngr
import ce_reference as C
import join_reference as J

pytestmark = pytest.mark.gpu
RMS, LAYER = 2, 1


@pytest.fixture(scope="module", autouse=True)
def _built():
    ngr.build()
    torch.cuda.init()


def chain(d, e, head, norm):
    """h0, y0 = join(x, residual); x1 = y0 W1^T; h1, y1 = join(x1, h0); the
    loss of y1; the gradients."""
    kw0 = dict(gate=d["gate"], norm1=norm, gamma1=d["gamma1"], beta1=d["beta1"], norm2=norm, gamma2=d["gamma2"], beta2=d["beta2"])
    kw1 = dict(gate=e["gate"], norm1=norm, gamma1=e["gamma1"], beta1=e["beta1"], norm2=norm, gamma2=e["gamma2"], beta2=e["beta2"])
    o = {}
    o["h0"], o["y0"], o["s0"] = ngr.fused_norm_gate_residual_norm(d["x"], d["residual"], return_stats=True, **kw0)
    o["x1"] = ngr.fused_norm_linear_act(o["y0"], head["W1"])
    o["h1"], o["y1"], o["s1"] = ngr.fused_norm_gate_residual_norm(o["x1"], o["h0"], return_stats=True, **kw1)
    o["loss"], o["lse"] = ngr.fused_linear_cross_entropy(o["y1"], head["W"], head["target"])
    o["dy1"], o["dW"] = ngr.fused_linear_cross_entropy_backward(head["dloss"], o["lse"], o["y1"], head["W"], head["target"])
    # h1 goes nowhere else: its own gradient is zero
    o["g1"] = ngr.fused_norm_gate_residual_norm_backward(o["dy1"], None, o["x1"], o["h0"], o["s1"], **kw1)
    # (the product's own gradient is the caller's: here y0 feeds nothing else)
    o["g0"] = ngr.fused_norm_gate_residual_norm_backward(None, o["g1"]["dresidual"], d["x"], d["residual"], o["s0"], **kw0)
    return o


def inputs(M, N, V, dtype, norm, seed):
    d = J.case(M, N, norm, norm, 1, dtype, seed)
    e = J.case(M, N, norm, norm, 2, dtype, seed + 1)
    c = C.case(M, N, V, dtype, seed + 2, ignored=0.25)
    g = torch.Generator("cpu")
    g.manual_seed(seed + 3)
    c["W1"] = (torch.randn((N, N), generator=g) * N ** -0.5).to(dtype)
    return d, e, c


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("norm", [RMS, LAYER])
def test_every_step_of_the_chain(norm, dtype):
    M, N, V = 150, 256, 900
    d, e, c = inputs(M, N, V, dtype, norm, seed=5)
    cuda = lambda t: {k: (v.cuda() if v is not None else None) for k, v in t.items()}
    o = chain(cuda(d), cuda(e), cuda(c), norm)
    cpu = lambda t: t.cpu()

    j0 = dict(d, dy=None, dh=cpu(o["g1"]["dresidual"]))
    val, mag = J.reference(j0, norm, norm)
    for got, k in ((o["h0"], "h"), (o["y0"], "y"), (o["g0"]["dx"], "dx"), (o["g0"]["dresidual"], "dresidual"),
                   (o["g0"]["dgate"], "dgate"), (o["g0"]["dgamma1"], "dgamma1")):
        J.check(got, val[k], mag[k], dtype, f"first join {k}")
    assert (o["g0"]["dgamma2"] == 0).all()

    j1 = dict(e, x=cpu(o["x1"]), residual=cpu(o["h0"]), dy=cpu(o["dy1"]), dh=None)
    val, mag = J.reference(j1, norm, norm)
    for got, k in ((o["h1"], "h"), (o["y1"], "y"), (o["g1"]["dx"], "dx"), (o["g1"]["dresidual"], "dresidual"),
                   (o["g1"]["dgate"], "dgate"), (o["g1"]["dgamma1"], "dgamma1"), (o["g1"]["dgamma2"], "dgamma2")):
        J.check(got, val[k], mag[k], dtype, f"second join {k}")

    head = dict(c, x=cpu(o["y1"]))
    val, tol = C.reference(head, 1.0, c["dloss"])
    for got, k in ((o["loss"], "loss"), (o["lse"], "lse"), (o["dy1"], "dx"), (o["dW"], "dW")):
        C.check(got, val[k], tol[k], f"head {k}")
    # masked tokens: nothing comes back to them
    off = c["target"] < 0
    for g in (o["g1"]["dx"], o["g1"]["dresidual"], o["g0"]["dx"], o["g0"]["dresidual"]):
        assert (g.cpu()[off] == 0).all()


def test_captured_chain_follows_its_inputs():
    """One graph of the whole step, replayed on other inputs with another
    number of masked tokens, gives the bits of the calls made one by one."""
    M, N, V = 1300, 256, 1100
    sets = [inputs(M, N, V, torch.bfloat16, RMS, seed) for seed in (20, 30)]
    sets[1][2]["target"][: M // 2] = -1
    cuda = lambda t: {k: (v.cuda() if v is not None else None) for k, v in t.items()}
    live = [cuda(t) for t in sets[0]]
    chain(*live, RMS)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = chain(*live, RMS)
    for new in (1, 0):
        for held, given in zip(live, sets[new]):
            for k, v in given.items():
                if v is not None:
                    held[k].copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        got = {k: v.clone() for k, v in out.items() if torch.is_tensor(v)}
        got.update({f"g{i}{k}": v.clone() for i in (0, 1) for k, v in out[f"g{i}"].items() if v is not None})
        want = chain(*[cuda(t) for t in sets[new]], RMS)
        flat = {k: v for k, v in want.items() if torch.is_tensor(v)}
        flat.update({f"g{i}{k}": v for i in (0, 1) for k, v in want[f"g{i}"].items() if v is not None})
        for k, v in flat.items():
            assert torch.equal(got[k], v), k


def test_two_streams_at_once():
    """Two steps on two streams, each with workspaces of its own, in turn
    many times: the bits of the same steps alone."""
    a, b = inputs(300, 512, 2000, torch.bfloat16, RMS, 40), inputs(700, 512, 1500, torch.bfloat16, RMS, 50)
    cuda = lambda t: {k: (v.cuda() if v is not None else None) for k, v in t.items()}
    a, b = [cuda(t) for t in a], [cuda(t) for t in b]
    want = [chain(*a, RMS), chain(*b, RMS)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [None, None]
    for _ in range(5):
        for i, t in enumerate((a, b)):
            with torch.cuda.stream(streams[i]):
                got[i] = chain(*t, RMS)
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        for k in ("loss", "dy1", "dW", "h1"):
            assert torch.equal(w[k], g[k]), k
        assert torch.equal(w["g0"]["dx"], g["g0"]["dx"]) and torch.equal(w["g1"]["dgate"], g["g1"]["dgate"])


def test_kernel_timing_counts_the_new_calls():
    from normalization_gemm_row_gb300 import binding as B
    a = [{k: (v.cuda() if v is not None else None) for k, v in t.items()} for t in inputs(200, 256, 600, torch.float16, RMS, 60)]
    chain(*a, RMS)
    B.kernel_timing_start(8)
    o = chain(*a, RMS)
    torch.cuda.synchronize()
    calls = B.kernel_timing_stop()
    # join 1; product; join 1; loss: gather, z, reduction; its gradient: the
    # first four kernels; the joins' gradients: rows, sums
    assert [len(c) for c in calls][0:1] + [len(c) for c in calls][2:] == [1, 1, 3, 4, 2, 2]
    assert all(ms > 0 for c in calls for ms in c)
    assert torch.isfinite(o["loss"]).all()
