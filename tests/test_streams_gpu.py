"""The block join and the linear cross entropy launched on a stream that is
not the current one, whose memory the calls' tensors have to come from."""
import pytest
import torch

import normalization_gemm_row_gb300 as ngr
import ce_reference as C
import join_reference as J

pytestmark = pytest.mark.gpu
RMS = 2
LONG = 100_000_000       # clocks: tens of milliseconds


@pytest.fixture(scope="module", autouse=True)
def _built():
    ngr.build()
    torch.cuda.init()


def join_data():
    d = J.case(512, 1024, RMS, RMS, 1, torch.bfloat16, seed=1)
    return {k: (v.cuda() if v is not None else None) for k, v in d.items()}


def joins(c, stream=None):
    kw = dict(gate=c["gate"], norm1=RMS, gamma1=c["gamma1"], norm2=RMS, gamma2=c["gamma2"], stream=stream)
    h, y, st = ngr.fused_norm_gate_residual_norm(c["x"], c["residual"], return_stats=True, **kw)
    g = ngr.fused_norm_gate_residual_norm_backward(c["dy"], c["dh"], c["x"], c["residual"], st, **kw)
    return [h, y, st] + [g[k] for k in ("dx", "dresidual", "dgate", "dgamma1", "dgamma2")]


def ce_data():
    return {k: v.cuda() for k, v in C.case(512, 1024, 1024, torch.bfloat16, seed=2, ignored=0.2).items()}


def losses(c, stream=None):
    loss, lse = ngr.fused_linear_cross_entropy(c["x"], c["W"], c["target"], stream=stream)
    return [loss, lse, *ngr.fused_linear_cross_entropy_backward(c["dloss"], lse, c["x"], c["W"], c["target"], stream=stream)]


CALLS = [(join_data, joins), (ce_data, losses)]


@pytest.mark.parametrize("data,call", CALLS)
def test_memory_that_the_current_stream_still_reads(data, call):
    """Blocks freed on the current stream while its copies out of them wait
    behind other work: the call on another stream writes into none of them."""
    c = data()
    want = call(c)
    side = torch.cuda.Stream()
    # blocks of the results' sizes, of the workspaces' among them
    sizes = [t.numel() * t.element_size() for t in want] * 2 + [1 << 20, 2 << 20, 4 << 20] * 2
    copies = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes]
    del want
    blocks = [torch.full((n,), 7, dtype=torch.uint8, device="cuda") for n in sizes]
    torch.cuda.synchronize()
    torch.cuda._sleep(LONG)
    for a, b in zip(copies, blocks):
        a.copy_(b)
    del blocks, a, b
    got = call(c, side)
    side.synchronize()
    torch.cuda.synchronize()
    for a in copies:
        assert (a == 7).all()
    for a, b in zip(got, call(c)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("data,call", CALLS)
def test_results_that_the_current_stream_still_reads(data, call):
    """Results of a call on another stream, freed while the current stream's
    copies of them wait: the next call there does not write over them."""
    c = data()
    want = call(c)
    side = torch.cuda.Stream()
    got = call(c, side)
    side.synchronize()
    copies = [torch.empty_like(t) for t in got]
    other = {k: (v * 0 if v is not None and v.is_floating_point() else v) for k, v in c.items()}
    torch.cuda.synchronize()
    torch.cuda._sleep(LONG)
    for a, b in zip(copies, got):
        a.copy_(b)
    del got, a, b
    for _ in range(3):
        call(other, side)
    torch.cuda.synchronize()
    for a, b in zip(copies, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("data,call", CALLS)
def test_streams_as_objects_and_handles(data, call):
    c = data()
    want = call(c)
    torch.cuda.synchronize()
    side, inner = torch.cuda.Stream(), torch.cuda.Stream()
    for given in (side, side.cuda_stream, torch.cuda.default_stream(), 0):
        for outer in (torch.cuda.default_stream(), inner, side):
            with torch.cuda.stream(outer):
                got = call(c, given)
                assert torch.cuda.current_stream() == outer
            torch.cuda.synchronize()
            for a, b in zip(got, want):
                assert torch.equal(a, b)


def test_launched_on_the_stream_that_is_given():
    """The work is the given stream's, however it is named: an event of
    that stream is not done before the sleep ahead of it is."""
    c = join_data()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for given, stream in ((side, side), (side.cuda_stream, side), (0, torch.cuda.default_stream())):
        with torch.cuda.stream(torch.cuda.Stream()):
            h = torch.zeros_like(c["x"])
            torch.cuda.current_stream().synchronize()
            with torch.cuda.stream(stream):
                torch.cuda._sleep(LONG)
            ngr.fused_norm_gate_residual_norm(c["x"], c["residual"], norm1=0, norm2=0, h=h, stream=given)
            seen = h.clone()
            torch.cuda.current_stream().synchronize()
            assert (seen == 0).all()
            stream.synchronize()
            assert not (h == 0).all()


@pytest.mark.parametrize("data,call", CALLS)
def test_another_stream_within_a_capture(data, call):
    c = data()
    want = call(c)
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        got = call(c, side)
        torch.cuda.current_stream().wait_stream(side)
    for _ in range(2):
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_refusals_are_the_same_on_another_stream():
    c = ce_data()
    side = torch.cuda.Stream()
    for stream in (None, side):
        for workspace in (torch.empty(1 << 24, dtype=torch.uint8), torch.empty(256, dtype=torch.uint8, device="cuda")):
            with pytest.raises(ValueError, match="workspace"):
                ngr.fused_linear_cross_entropy(c["x"], c["W"], c["target"], workspace=workspace, stream=stream)
        with pytest.raises(ValueError, match="one entry"):
            ngr.fused_linear_cross_entropy(c["x"], c["W"], c["target"][:-1], stream=stream)
        with pytest.raises(ngr.NgrError):
            ngr.fused_linear_cross_entropy(c["x"], c["W"], c["target"], logit_scale=float("nan"), stream=stream)
        assert torch.cuda.current_stream() == torch.cuda.default_stream()
