"""A process whose first calls are made inside a capture, and calls from
several threads at once."""
import os
import subprocess
import sys
import threading

import pytest
import torch

import normalization_gemm_row_gb300 as ngr
import test_streams_gpu as S

pytestmark = pytest.mark.gpu

CHILD = r"""
import sys
sys.path.insert(0, "tests")
import torch
import test_streams_gpu as S
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


@pytest.mark.parametrize("which", [0, 1])
def test_first_call_inside_a_capture(which):
    ngr.build()
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    p = subprocess.run([sys.executable, "-c", CHILD, str(which)], cwd=root, capture_output=True, text=True, timeout=300)
    assert p.returncode == 0, p.stderr
    assert p.stdout.strip() == "same"


def test_threads():
    torch.cuda.init()
    data = [(d(), call) for d, call in S.CALLS * 2]
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
