"""The rotated append, the paged attention and the experts on streams that are
not the current one, in captures, threads and processes of their own."""
import os
import re
import subprocess
import sys
import threading

import pytest
import torch

import normalization_gemm_row_gb300 as ngr
import kv_reference as K
import moe_reference as M
import test_streams_gpu as S

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _built():
    ngr.build()
    torch.cuda.init()


def append_data():
    g = K.generator(1)
    T, H, G, D = 64, 8, 4, 64
    c = {n: torch.randn((T, h, D), generator=g).to(F16) for n, h in (("q", H), ("k", G), ("v", G))}
    c["table"], pages = K.pages_for([90] * T, 16, g)
    c["positions"] = torch.randint(0, 90, (T,), generator=g, dtype=torch.int32)
    c["inv"] = (10000.0 ** (-torch.arange(0, D, 2, dtype=torch.float64) / D)).float()
    c["kc"], c["vc"] = torch.zeros((pages, 16, G, D), dtype=F16), torch.zeros((pages, 16, G, D), dtype=F16)
    return {n: t.cuda() for n, t in c.items()}


def append(c, stream=None):
    q = ngr.fused_rope_append_kv(c["q"], c["k"], c["v"], c["kc"], c["vc"], c["table"], c["positions"], inv_freq=c["inv"], stream=stream)
    return [q]


def attend_data(lengths=tuple(range(0, 900, 10))):
    g = K.generator(2)
    c = {"q": torch.randn((len(lengths), 8, 64), generator=g).to(BF16)}
    c["table"], pages = K.pages_for(list(lengths), 16, g)
    c["kc"], c["vc"] = (torch.randn((pages, 16, 2, 64), generator=g).to(BF16) for _ in range(2))
    c["lengths"] = torch.tensor(lengths, dtype=torch.int32)
    return {n: t.cuda() for n, t in c.items()}


def attend(c, stream=None):
    return list(ngr.fused_paged_attention(c["q"], c["kc"], c["vc"], c["table"], c["lengths"], return_lse=True, stream=stream))


def moe_data():
    d = M.separate(M.case(9, 256, 320, 12, BF16, 3), 3)
    return {n: t.cuda() for n, t in d.items() if t is not None}


def experts(c, stream=None):
    return list(ngr.fused_moe_swiglu(c["x"], c["Wr"], c["Wg"], c["Wu"], c["Wd"], 3, norm=2, gamma=c["gamma"], return_routing=True,
                                     stream=stream))


CALLS = [(append_data, append), (attend_data, attend), (lambda: attend_data((3, 100, 0)), attend), (moe_data, experts)]


@pytest.mark.parametrize("data,call", CALLS)
def test_memory_that_the_current_stream_still_reads(data, call):
    S.test_memory_that_the_current_stream_still_reads(data, call)


@pytest.mark.parametrize("data,call", CALLS[:1] + CALLS[3:])
def test_results_that_the_current_stream_still_reads(data, call):
    S.test_results_that_the_current_stream_still_reads(data, call)


@pytest.mark.parametrize("data,call", CALLS)
def test_streams_as_objects_and_handles(data, call):
    S.test_streams_as_objects_and_handles(data, call)


@pytest.mark.parametrize("data,call", CALLS)
def test_another_stream_within_a_capture(data, call):
    S.test_another_stream_within_a_capture(data, call)


def test_threads():
    data = [(d(), call) for d, call in CALLS * 2]
    want = [call(c) for c, call in data]
    torch.cuda.synchronize()
    bad = []

    def work(i):
        c, call = data[i]
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(20):
                got = call(c)
                torch.cuda.current_stream().synchronize()
                if not all(torch.equal(a, b) for a, b in zip(got, want[i])):
                    bad.append(i)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(data))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad


CHILD = r"""
import sys
sys.path.insert(0, "tests")
import torch
import test_step_streams_gpu as S
data, call = S.CALLS[int(sys.argv[1])]
c = data()
graph = torch.cuda.CUDAGraph()
torch.cuda.synchronize()
with torch.cuda.graph(graph):
    got = call(c)
graph.replay()
torch.cuda.synchronize()
print("same" if all(torch.equal(a, b) for a, b in zip(got, call(c))) else "not the same")
"""


@pytest.mark.parametrize("which", [0, 1, 2, 3])
def test_first_call_inside_a_capture(which):
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    p = subprocess.run([sys.executable, "-c", CHILD, str(which)], cwd=root, capture_output=True, text=True, timeout=300)
    assert p.returncode == 0, p.stderr
    assert p.stdout.strip() == "same"


TRACED = r"""
import sys
sys.path.insert(0, "tests")
import torch
import normalization_gemm_row_gb300 as ngr
import test_step_streams_gpu as S
for data, call in S.CALLS:
    call(data())
torch.cuda.synchronize()
# bad pages: reported by the call itself with NGR_DEBUG
for data, call in S.CALLS[:3]:
    c = data()
    c["table"].fill_(10 ** 6)
    try:
        call(c)
        torch.cuda.synchronize()
        print("passed")
    except ngr.NgrError as e:
        print("reported", e.status)
"""
LINES = [r"ngr: rotated append T=64 H=8 G=4 D=64 rot=64 page=16 elements at once=8 blocks a token=\d+",
         r"ngr: paged attention B=90 H=8 G=2 D=64 page=16 window=0 dim=64 workers=\d+ jobs=\d+",
         r"ngr: paged attention B=3 H=8 G=2 D=64 page=16 window=0 dim=64 items=6 jobs=0",
         r"ngr: experts M=9 K=256 F=320 E=12 top_k=3 norm=2 groups=2"]


def test_trace_and_debug():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    for on in ("1", "0"):
        p = subprocess.run([sys.executable, "-c", TRACED], cwd=root, env=dict(os.environ, NGR_TRACE=on, NGR_DEBUG=on), capture_output=True,
                           text=True, timeout=300)
        assert p.returncode == 0, p.stderr
        got = [line for line in p.stderr.split("\n") if line.startswith("ngr: ")]
        assert len(got) == (len(LINES) + 3 if on == "1" else 0), p.stderr
        for a, b in zip(got, LINES):
            assert re.fullmatch(b, a), (a, b)
        assert p.stdout.split("\n")[:3] == ["reported -9" if on == "1" else "passed"] * 3
