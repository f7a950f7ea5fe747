"""The rotated append in calls large enough for several heads a thread: every
element written, every other one untouched (the check of test_append_gpu.py)."""
import pytest
import torch

import normalization_gemm_row_gb300 as ngr
from test_append_gpu import run

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16
MANY = 2 * 152 * 2048      # units (pairs of accesses) of a call from which a thread takes four heads


@pytest.fixture(scope="module", autouse=True)
def _built():
    ngr.build()
    torch.cuda.init()


def units(vec, interleaved, D, rot):
    """Units of a head that is moved by accesses of vec elements."""
    up = lambda n: -(-n // (2 * vec))
    turned = up(D) if interleaved and vec > 1 else rot // 2 // vec + up(D - rot)
    return max(turned, up(D))


def large(H, G, D, dtype, vec, rot=None, interleaved=False, below=False, **kw):
    rot = D if rot is None else rot
    per_token = (H + 2 * G) * units(vec, interleaved, D, rot)
    T = (MANY - 1) // per_token if below else -(-MANY // per_token)
    assert (T * per_token >= MANY) != below
    # tokens of two sequences, some left out
    positions = [t // 2 if t % 7 else -1 for t in range(T)]
    run(T, H, G, D, 64, dtype, rot=rot, interleaved=interleaved, positions=positions, rows=[t % 2 for t in range(T)], sequences=2, **kw)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("vec,offset", [(8, 0), (4, 4), (2, 2), (1, 1)])
def test_accesses_of_every_size(vec, offset, interleaved, dtype):
    """(10 + 2 x 5 heads of 80: no multiple of the heads that a block takes)"""
    large(10, 5, 80, dtype, vec, interleaved=interleaved, offset=offset, layout="tokens" if vec == 8 else "wide")


@pytest.mark.parametrize("H,G,D", [(64, 8, 128), (71, 1, 128), (1, 1, 64), (7, 7, 96), (3, 2, 256), (33, 4, 192)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_heads(H, G, D, interleaved):
    large(H, G, D, BF16, 8, interleaved=interleaved, layout="heads")


@pytest.mark.parametrize("D,rot,vec", [(128, 64, 8), (80, 32, 8), (80, 20, 2), (64, 0, 8), (72, 24, 4), (5, 4, 1), (2, 2, 1)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_partial_rotation(D, rot, vec, interleaved):
    if interleaved and rot % 8 and vec > 1:
        vec = rot & -rot
    elif interleaved and vec > 1:
        vec = 8
    large(6, 3, D, F16, vec, rot=rot, interleaved=interleaved)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("vec,offset", [(8, 0), (2, 2)])
def test_in_place(vec, offset, interleaved):
    large(10, 5, 80, BF16, vec, interleaved=interleaved, in_place=True, offset=offset)


@pytest.mark.parametrize("interleaved", [False, True])
def test_one_call_less(interleaved):
    """Just below the size: a head a thread."""
    large(10, 5, 80, F16, 8, interleaved=interleaved, below=True)
