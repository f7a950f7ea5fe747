"""A decode step as it is used: the QKV product with its norm, the rotated
append, attention over the cache, the output product with residual and norm,
and a mixture-of-experts layer, for a batch whose sequences grow.

Each call is held to its formula in float64 on the inputs it was given (its
predecessors' outputs as stored)."""
import pytest
import torch

import normalization_gemm_row_gb300 as ngr
from normalization_gemm_row_gb300 import binding as B
import kv_reference as K
import moe_reference as M

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _built():
    ngr.build()
    torch.cuda.init()


class Block:
    """Weights, cache and buffers of one decoder block (CPU tensors and their copies on the GPU)."""

    def __init__(self, batch, dtype, seed, lengths, width=256, H=8, G=2, D=32, page=8, experts=6, F=96, room=4):
        g = K.generator(seed)
        self.dtype, self.H, self.G, self.D, self.page, self.batch, self.width = dtype, H, G, D, page, batch, width
        normal = lambda *s, std=1.0, mean=0.0: (torch.randn(s, generator=g) * std + mean).to(dtype)
        self.gamma = normal(width, std=0.1, mean=1.0)
        self.Wqkv = normal((H + 2 * G) * D, width, std=2.0 * width ** -0.5)
        self.Wo = normal(width, H * D, std=(H * D) ** -0.5)
        self.moe = M.case(batch, width, F, experts, dtype, seed + 1)
        self.inv = (10000.0 ** (-torch.arange(0, D, 2, dtype=torch.float64) / D)).float()
        self.table, pages = K.pages_for([n + 40 for n in lengths], page, g, room=room)
        self.k, self.v = (torch.randn((pages, page, G, D), generator=g).to(dtype) for _ in range(2))
        self.x = normal(batch, width)
        self.c = {n: getattr(self, n).cuda() for n in ("gamma", "Wqkv", "Wo", "inv", "table", "k", "v", "x")}
        self.c.update({n: self.moe[n].cuda() for n in ("Wr", "Wg", "Wu", "Wd")})
        self.positions = torch.tensor(lengths, dtype=torch.int32, device="cuda")      # of the token that comes now
        self.lengths = self.positions + 1

    def step(self, stream=None):
        c, H, G, D = self.c, self.H, self.G, self.D
        o = {}
        o["qkv"] = ngr.fused_rmsnorm_linear(c["x"], c["gamma"], c["Wqkv"], stream=stream)
        q, k, v = (o["qkv"][:, a * D:b * D].view(self.batch, -1, D) for a, b in ((0, H), (H, H + G), (H + G, H + 2 * G)))
        o["q"] = ngr.fused_rope_append_kv(q, k, v, c["k"], c["v"], c["table"], self.positions, inv_freq=c["inv"], stream=stream)
        o["o"], o["lse"] = ngr.fused_paged_attention(o["q"], c["k"], c["v"], c["table"], self.lengths, return_lse=True, stream=stream)
        o["h"], o["n"] = ngr.fused_linear_residual_norm(o["o"].view(self.batch, H * D), c["Wo"], c["gamma"], residual=c["x"], stream=stream)
        o["y"], o["experts"], o["weights"] = ngr.fused_moe_swiglu(o["h"], c["Wr"], c["Wg"], c["Wu"], c["Wd"], 2, norm=2, gamma=c["gamma"],
                                                                  return_routing=True, stream=stream)
        return o

    def check(self, o):
        o = {n: t.cpu() for n, t in o.items()}
        H, G, D = self.H, self.G, self.D
        q, k, v = (o["qkv"][:, a * D:b * D].reshape(self.batch, -1, D) for a, b in ((0, H), (H, H + G), (H + G, H + 2 * G)))
        pos = self.positions.cpu()
        used = pos >= 0
        kc, vc = self.c["k"].cpu(), self.c["v"].cpu()
        page = self.table[torch.arange(self.batch)[used], (pos[used] // self.page).long()].long()
        slot = (pos[used] % self.page).long()
        for got, given, what in ((o["q"][used], q, "q"), (kc[page, slot], k, "k")):
            val, mag = K.rotate(given.double(), pos.clamp(min=0), self.inv, False)
            K.check_rotated(got, val[used], mag[used], self.dtype, what)
        assert torch.equal(vc[page, slot], v[used])
        K.check_attention(o["o"], o["lse"], K.attention(o["q"], kc, vc, self.table, self.lengths.cpu(), D ** -0.5))
        d = dict(self.moe, x=o["h"], gamma=self.gamma)
        rows = used.nonzero()[:, 0]
        d["x"] = d["x"][rows]
        if M.apart(d, 2):      # (a choice that hangs on a rounding is no mistake)
            M.check((o["y"][rows], o["experts"][rows], o["weights"][rows]), M.reference(d, 2))


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_steps_of_a_growing_batch(dtype):
    b = Block(5, dtype, 1, [0, 7, 8, 30, 63])
    before = (b.c["k"].clone(), b.c["v"].clone())
    for _ in range(12):
        b.check(b.step())
        b.positions += 1
        b.lengths += 1
    # only the twelve new slots of each sequence have changed
    fresh = torch.zeros(b.k.shape[:2], dtype=torch.bool)
    for r, n in enumerate([0, 7, 8, 30, 63]):
        j = torch.arange(n, n + 12)
        fresh[b.table[r].long()[j // b.page], j % b.page] = True
    for new, old in zip((b.c["k"], b.c["v"]), before):
        assert torch.equal(new.cpu()[~fresh], old.cpu()[~fresh])


def test_rows_of_a_padded_batch():
    """Rows behind the last sequence: position and length below zero.  Nothing of them is appended; what the other
    rows get is what they get without them."""
    b = Block(6, F16, 2, [3, 11, 20, 5, 9, 1])
    b.positions[3:] = -1
    b.lengths[3:] = -1
    k, v = b.c["k"].clone(), b.c["v"].clone()
    o = b.step()
    b_k = b.c["k"].clone()
    b.c["k"].copy_(k)
    b.c["v"].copy_(v)
    c = b.c
    q = o["qkv"][:3, :b.H * b.D].view(3, b.H, b.D)
    kk = o["qkv"][:3, b.H * b.D:(b.H + b.G) * b.D].view(3, b.G, b.D)
    vv = o["qkv"][:3, (b.H + b.G) * b.D:].view(3, b.G, b.D)
    q2 = ngr.fused_rope_append_kv(q, kk, vv, c["k"], c["v"], c["table"][:3], b.positions[:3], inv_freq=c["inv"])
    o2 = ngr.fused_paged_attention(q2, c["k"], c["v"], c["table"][:3], b.lengths[:3])
    assert torch.equal(q2, o["q"][:3]) and torch.equal(b_k, c["k"]) and torch.equal(o2, o["o"][:3])


def same(a, b):
    return all(torch.equal(a[n], b[n]) for n in a)


def test_captured_step_follows_positions_and_lengths():
    """One graph, replayed while the sequences grow and shrink, gives the bits of the calls made one by one."""
    b, e = (Block(7, BF16, 3, [0, 7, 8, 30, 63, 2, 17]) for _ in range(2))
    b.step()
    torch.cuda.synchronize()
    b.c["k"].copy_(e.c["k"])
    b.c["v"].copy_(e.c["v"])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = b.step()
    for positions in ([0, 7, 8, 30, 63, 2, 17], [1, 8, 9, 31, 64, 3, 18], [38, 0, -1, 12, 5, -1, 50], [39, 1, 0, 13, 6, 3, 51]):
        for x in (b, e):
            x.positions.copy_(torch.tensor(positions))
            x.lengths.copy_(torch.tensor([p + 1 if p >= 0 else -1 for p in positions]))
        for t in out.values():
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        want = e.step()
        used = torch.tensor([p >= 0 for p in positions], device="cuda")
        for n in ("q", "o", "lse", "h", "n", "y", "experts", "weights"):
            assert torch.equal(out[n][used], want[n][used]), n
        assert torch.equal(b.c["k"], e.c["k"]) and torch.equal(b.c["v"], e.c["v"])


def test_two_graphs_of_one_workspace_in_turn():
    """Two captured calls with one workspace, replayed in any order on one stream."""
    small, large = Block(2, F16, 4, [9, 30]), Block(40, F16, 5, [50] * 40)
    n = max(B.ngr_paged_attention_workspace_bytes(x.batch, x.H, x.G, x.D, x.table.shape[1] * x.page, 0) for x in (small, large))
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    graphs, outs, want, held = [], [], [], []
    for x in (small, large):
        q = torch.randn((x.batch, x.H, x.D), generator=K.generator(6)).to(F16).cuda()
        args = (q, x.c["k"], x.c["v"], x.c["table"], x.lengths)
        held.append(args)
        want.append(ngr.fused_paged_attention(*args))
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(ngr.fused_paged_attention(*args, workspace=ws))
        graphs.append(g)
    for i in (0, 1, 1, 0, 0, 1):
        outs[i].zero_()
        graphs[i].replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[i], want[i])


def test_two_streams_at_once():
    blocks = [Block(4, BF16, 7, [100, 3, 50, 20]), Block(9, BF16, 8, [60] * 9)]
    want = [x.step() for x in blocks]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [None, None]
    for _ in range(10):
        for i, x in enumerate(blocks):
            with torch.cuda.stream(streams[i]):
                got[i] = x.step()
    torch.cuda.synchronize()
    assert same(want[0], got[0]) and same(want[1], got[1])


@pytest.mark.parametrize("batch,room,kernels", [(3, 4, 1), (3, 400, 2), (100, 4, 2)])
def test_kernel_timing_and_launches(batch, room, kernels):
    """Short tables of few sequences take one kernel, others two; append one, experts three."""
    x = Block(batch, F16, 9, [5] * batch, room=room)
    q = torch.randn((batch, x.H, x.D)).to(F16).cuda()
    kv = torch.randn((batch, x.G, x.D)).to(F16).cuda()
    c = x.c
    B.kernel_timing_start(3)
    ngr.fused_rope_append_kv(q, kv, kv, c["k"], c["v"], c["table"], x.positions, inv_freq=c["inv"])
    ngr.fused_paged_attention(q, c["k"], c["v"], c["table"], x.lengths)
    ngr.fused_moe_swiglu(c["x"][:32], c["Wr"], c["Wg"], c["Wu"], c["Wd"], 2, norm=2, gamma=c["gamma"])
    torch.cuda.synchronize()
    calls = B.kernel_timing_stop()
    assert [len(t) for t in calls] == [1, kernels, 3]
    assert all(ms > 0 for t in calls for ms in t)
