"""How the block join's kernels cut a row into CTAs, for every width, way of
reaching the row and number of column sums: the cluster that a launch asks for
has to be one that the kernels have room for and the device can give."""
import ctypes

import pytest

import normalization_gemm_row_gb300 as pkg
from normalization_gemm_row_gb300 import binding as B

ALIGNED, WINDOW, SCALAR = 0, 1, 2
MAX_N = 65536
MAX_CLUSTER = 16          # the largest cluster of sm_103
THREADS, VECTORS = 512, {"forward": 5, "backward": 2}      # (five: a row of one warp)


class Shape(ctypes.Structure):
    _fields_ = [(k, ctypes.c_int) for k in ("cluster", "cols", "vecs", "tpr", "slots", "per_sm")]


@pytest.fixture(scope="module")
def shapes():
    pkg.build()
    lib = B.lib()
    forward, backward = lib._ZN3ngr18join_forward_shapeEli, lib._ZN3ngr19join_backward_shapeElii
    forward.restype = backward.restype = Shape
    forward.argtypes = [ctypes.c_int64, ctypes.c_int]
    backward.argtypes = [ctypes.c_int64, ctypes.c_int, ctypes.c_int]
    return forward, backward


def covers(s, N, mode, vectors):
    assert s.cluster & (s.cluster - 1) == 0 and s.cols % 8 == 0
    assert s.cluster * s.cols >= N > (s.cluster - 1) * s.cols        # no CTA without a column
    assert s.tpr * s.vecs >= s.cols // 8 + (mode == WINDOW)          # a vector for each of them
    assert s.tpr % 32 == 0 and s.tpr <= THREADS and s.vecs <= vectors
    assert s.slots >= 1 and s.tpr * s.slots <= THREADS and (s.slots == 1 or s.cluster == 1)


@pytest.mark.parametrize("mode", [ALIGNED, WINDOW, SCALAR])
def test_every_width_has_its_ctas(shapes, mode):
    forward, backward = shapes
    widths = [n for n in range(1, MAX_N + 1) if mode != ALIGNED or n % 8 == 0]
    for N in widths[::7] + widths[-5000:]:
        s = forward(N, mode)
        assert s.cluster <= 8, (N, s.cluster)
        covers(s, N, mode, VECTORS["forward"])
    for sums in range(6):
        for N in widths[::29] + widths[-4500:]:
            s = backward(N, mode, sums)
            assert s.cluster <= MAX_CLUSTER and s.per_sm >= 1, (N, sums, s.cluster)
            covers(s, N, mode, VECTORS["backward"])
            # the sums of the CTAs of an SM, and a row each, in its shared memory
            cols = s.cols + 16 if mode == WINDOW else s.cols
            row = (4 * s.vecs + 1) * s.tpr * s.slots * 16
            # (2 KB a CTA for the sums over a row, 1 KB that the device takes)
            assert s.per_sm * (sums * s.slots * cols * 4 + row + 3 * 1024) <= 228 * 1024, (N, sums)


def test_widest_rows_are_sized():
    f = B.ngr_norm_gate_residual_norm_workspace_bytes
    for N in (61313, 61440, 61448, 65472, 65473, 65535, 65536):
        for rows_per_gate in (0, 1, 3, 16):
            assert f(1, 1, rows_per_gate, 48, N) > 256


def test_every_compiled_width_is_taken(shapes):
    """(threads on a row, vectors a thread, whether a CTA has whole rows):
    what the launches list, and nothing that no width leads to."""
    one = [(32, 1), (32, 2), (96, 1), (64, 2), (160, 1), (96, 2), (128, 2), (192, 2), (256, 2), (384, 2), (512, 2)]
    for mode in (ALIGNED, WINDOW, SCALAR):
        widths = range(8, MAX_N + 1, 8) if mode == ALIGNED else range(1, MAX_N + 1, 3)
        taken = lambda f: {(s.tpr, s.vecs, s.cluster == 1) for s in map(f, widths)}
        got = taken(lambda n: shapes[0](n, mode))
        want = {(512, 4, True), (512, 4, False), (256, 4, True)}
        if mode != SCALAR:
            want |= {(32, v, True) for v in range(1, 6)} | {(t, v, True) for t in (64, 128) for v in (3, 4)}
            want |= {(256, 3, True), (512, 3, True), (512, 3, False)}
        assert got == want
        # without a LayerNorm three sums at most, with one five
        for most in (3, 5):
            got = set().union(*(taken(lambda n: shapes[1](n, mode, k)) for k in range(most + 1)))
            want = {(64, 2, True), (512, 2, True), (512, 2, False)}
            if mode != SCALAR:
                want |= {(*w, True) for w in one} | {(384, 2, False)} | ({(256, 2, False)} if most == 5 else set())
            assert got == want, (mode, most)
