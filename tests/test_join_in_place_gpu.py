"""The block join's outputs in its inputs' memory, forward and gradient,
aligned, unaligned (where rows share 16-byte words), element by element and in
clusters: the same bits as apart, and nothing else written."""
import pytest
import torch

import normalization_gemm_row_gb300 as ngr
from normalization_gemm_row_gb300 import binding as B
import join_reference as R
import test_join_gpu as J

pytestmark = pytest.mark.gpu
LAYER, RMS = J.LAYER, J.RMS


@pytest.fixture(scope="module", autouse=True)
def _built():
    ngr.build()
    torch.cuda.init()


class Framed:
    """A tensor inside a buffer of sevens, `off` elements behind a 16-byte
    boundary."""
    def __init__(self, t, off):
        self.whole = torch.full((t.numel() + 64,), 7.0, dtype=t.dtype, device="cuda")
        self.t = self.whole[32 + off:32 + off + t.numel()].view(t.shape)
        self.t.copy_(t)
        self.ends = (self.whole[:32 + off], self.whole[32 + off + t.numel():])

    def intact(self):
        return all((e == 7.0).all() for e in self.ends)


def ptr(t):
    return None if t is None else t.data_ptr()


@pytest.mark.parametrize("offsets", [(0, 0, 0, 0), (3, 3, 3, 3), (0, 1, 2, 5)])
@pytest.mark.parametrize("M,N,gates", [(700, 1152, 1), (2000, 75, 2), (613, 2048, 0), (500, 1157, 500), (40, 8203, 4), (9, 20000, 0)])
def test_outputs_in_the_inputs_memory(M, N, gates, offsets):
    for norm in (LAYER, RMS):
        c = J.cuda(R.case(M, N, norm, norm, gates, torch.bfloat16, seed=M + N))
        args = J.how(c, norm, norm)
        place = lambda: {k: Framed(c[k], o) for k, o in zip(("x", "residual", "dy", "dh"), offsets)}
        # apart, from the same addresses' alignment
        f = place()
        h, y, st = ngr.fused_norm_gate_residual_norm(f["x"].t, f["residual"].t, return_stats=True,
                                                     h=Framed(c["x"], offsets[1]).t, out=Framed(c["x"], offsets[0]).t, **args)
        n = B.ngr_norm_gate_residual_norm_workspace_bytes(norm, norm, M // gates if gates else 0, M, N)
        ws = torch.empty(n, dtype=torch.uint8, device="cuda")
        s = torch.cuda.current_stream().cuda_stream

        def gradient(f, dx, dr):
            dg = torch.empty_like(c["gate"]) if gates else None
            v = [torch.empty_like(c["gamma1"]) for _ in range(4)]
            assert B.ngr_fused_norm_gate_residual_norm_backward(
                norm, norm, ptr(f["dy"].t), ptr(f["dh"].t), ptr(f["x"].t), ptr(f["residual"].t), ptr(c["gate"]),
                M // gates if gates else 0, ptr(c["gamma1"]), ptr(c["beta1"]), ptr(c["gamma2"]), ptr(st), 1.0, 1.0, M, N, 1,
                ptr(dx), ptr(dr), ptr(dg), *[ptr(t) for t in v], ptr(ws), n, s) == 0
            return [dx, dr, dg] + v[:4 if norm == LAYER else 3:1 if norm == LAYER else 2]

        for a, b in (("x", "residual"), ("residual", "dy"), ("dy", "dh"), ("dh", "x")):
            at = {k: o for k, o in zip(("x", "residual", "dy", "dh"), offsets)}
            want = gradient(f, Framed(c["x"], at[a]).t, Framed(c["x"], at[b]).t)
            g = place()
            got = gradient(g, g[a].t, g[b].t)
            for k, (p, q) in enumerate(zip(got, want)):
                assert p is None or torch.equal(p, q), (norm, a, b, k)
            assert all(v.intact() for v in g.values())
        for a, b in (("x", "residual"), ("residual", "x")):
            g = place()
            hh, yy = ngr.fused_norm_gate_residual_norm(g["x"].t, g["residual"].t, h=g[a].t, out=g[b].t, **args)
            # (with arrays at different places either order is element by element)
            assert torch.equal(hh, h) and torch.equal(yy, y), (norm, a, b)
            assert all(v.intact() for v in g.values())
