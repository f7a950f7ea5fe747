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
    """Weights of the other tokens that are all half a step above a power of two (a little less): two parts hold them;
    one part would take their sum half a step down."""
    score = -math.log((1 + 0.98 * R.U[dtype]) / 32)
    one_and_many(n, at, D, score, dtype, rows, B.two_parts(dtype), f"{n} tokens")


@pytest.mark.parametrize("lengths", [[100, 33], [3000, 1] + [200] * 150, [90000]])
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("D", [64, 80, 256])
def test_infinite_values(lengths, dtype, D):
    """An infinite value is its dimension's result, for every head and whatever the token's weight; both signs are NaN;
    the other dimensions are as they were."""
    g = R.generator(D)
    table, pages = R.pages_for(lengths, 16, g)
    k, v = R.cache_like(pages, 16, 2, D, dtype, "tokens", g)
    q = torch.randn((len(lengths), 8, D), generator=g).to(dtype)
    n = torch.tensor(lengths, dtype=torch.int32)
    want = R.attention(q, k, v, table, n, D ** -0.5)
    wild = [3, 17, 40]
    for b, size in enumerate(lengths):
        for at in {0, size // 3, size - 1}:
            page = table[b, at // 16]
            v[page, at % 16, :, 3] = float("inf")
            v[page, at % 16, :, 17] = -float("inf")
            v[page, at % 16, :, 40] = float("inf") if at else -float("inf")
    out = ngr.fused_paged_attention(q.cuda(), k.cuda(), v.cuda(), table.cuda(), n.cuda()).cpu()
    assert (out[..., 3] == float("inf")).all() and (out[..., 17] == -float("inf")).all()
    several = n > 3
    assert torch.isnan(out[several][..., 40]).all()
    tame = [d for d in range(D) if d not in wild]
    assert ((out.double() - want[0]).abs() <= want[2])[..., tame].all()


@pytest.mark.parametrize("n,rows", [(1000, 2), (8192, 2600), (60000, 1)])
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("far", ["infinitely", "beyond the smallest weight"])
def test_tokens_without_weight_have_none(n, rows, dtype, far):
    """Keys whose score is -inf, or 100 below the others', with fp16's largest values: nothing of them counts."""
    page, D = 64, 64
    pages = -(-n // page)
    k = torch.zeros((pages, page, 1, D), dtype=dtype)
    k[..., 0] = -float("inf") if far == "infinitely" else -100
    v = torch.full((pages, page, 1, D), 65504.0, dtype=dtype)
    few = torch.linspace(0.5, 2, D).to(dtype)
    for at in (0, n // 3, n - 1):
        k[at // page, at % page, 0, 0] = 0
        v[at // page, at % page, 0] = few
    q = torch.zeros((rows, 2, D), dtype=dtype)
    q[..., 0] = 1
    table = torch.arange(pages, dtype=torch.int32).repeat(rows, 1)
    lengths = torch.full((rows,), n, dtype=torch.int32)
    out, lse = ngr.fused_paged_attention(q.cuda(), k.cuda(), v.cuda(), table.cuda(), lengths.cuda(), scale=1.0, return_lse=True)
    # three weights of 1, each off by 3 x 2^-15 (fp16 2^-21) at most and alike, whose sum is divided by 3 and rounded
    # (e^-100 x 65504 x n is below 1e-33)
    want = few.double()
    assert ((out.double().cpu() - want).abs() <= (R.U[dtype] + B.two_parts(dtype) + 2.0 ** -21) * want).all()
    assert ((lse.cpu() - math.log(3)).abs() <= 2.0 ** -20).all()
