"""Paged attention where the softmax weights' own precision decides: many small
ones beside a large one, many that are equal."""
import math

import pytest
import torch

import normalization_gemm_row_gb300 as ngr
import kv_bounds as B
import kv_reference as R

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _built():
    ngr.build()
    torch.cuda.init()


def one_and_many(n, at, D, score, dtype, rows, weight, what):
    """n tokens of score 0 and equal values, but for token `at` of the given score and value 0; all rows of the batch
    have the same pages."""
    page = 64
    pages = -(-n // page)
    k = torch.zeros((pages, page, 1, D), dtype=dtype)
    v = torch.linspace(0.75, 1.5, D).to(dtype).repeat(pages, page, 1, 1)
    k[at // page, at % page, 0, 0] = 1
    v[at // page, at % page] = 0
    q = torch.zeros((rows, 2, D), dtype=dtype)
    q[:, :, 0] = 1
    table = torch.arange(pages, dtype=torch.int32).repeat(rows, 1)
    lengths = torch.full((rows,), n, dtype=torch.int32)
    out, lse = ngr.fused_paged_attention(q.cuda(), k.cuda(), v.cuda(), table.cuda(), lengths.cuda(), scale=score, return_lse=True)
    flat = [t.double().view(-1, D)[:n] for t in (k, v)]
    want, want_lse, tol = B.attention(q[0, 0].double(), *flat, score, dtype, weight, runs=64)
    r = ((out.double().cpu() - want).abs() / tol).max().item()
    assert r <= 1, f"{what}: worst {r:.2f} times the tolerance"
    assert ((lse.double().cpu() - want_lse).abs() <= 2.0 ** -17 * (1 + score)).all()


# (a CTA takes a row alone; several rows to a worker; several workers to a row)
SHAPES = [(1000, 3, 2), (3000, 40, 3000), (27000, 5, 1)]


@pytest.mark.parametrize("n,at,rows", SHAPES)
@pytest.mark.parametrize("score", [10.4, 14.2, 17.3, 20.0])
@pytest.mark.parametrize("D", [64, 128])
def test_many_small_weights_in_fp16(n, at, rows, score, D):
    """Weights down to e^-20 of the largest keep their share: each is off by at most half a step of fp16, relative."""
    one_and_many(n, at, D, score, F16, rows, R.U[F16], f"{n} tokens")


@pytest.mark.parametrize("n,at,rows", SHAPES)
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("D", [64, 80, 256])
def test_equal_weights_between_two_steps(n, at, rows, dtype, D):
    """Weights of the other tokens that are all half a step above a power of two (a little less): two parts hold them,
    each off by half a step of half a step; one part would take their sum half a step down."""
    score = -math.log((1 + 0.98 * R.U[dtype]) / 32)
    one_and_many(n, at, D, score, dtype, rows, R.U[dtype] ** 2, f"{n} tokens")
