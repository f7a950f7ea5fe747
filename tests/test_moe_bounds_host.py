"""The bound of moe_bounds.py against computations with a mistake in them: it
admits what the layer says it does and nothing less."""
import pytest
import torch

import moe_bounds as B
import moe_reference as R

F16, BF16 = torch.float16, torch.bfloat16


def two_parts(x, dtype):
    by, low = (256.0, 2048.0) if dtype is F16 else (1.0, 1.0)
    x = (x / by).float()
    hi = x.to(dtype)
    return (hi.double() + ((x - hi.float()) * low).to(dtype).double() / low) * by


def one_part(x, dtype):
    return x.to(dtype).double()


def layer(d, top_k, norm, a_parts, h_parts, lost_k=False, lost_f=False):
    """The layer in float64 with a and h rounded in this way, without the last column of K or of F."""
    dtype = d["x"].dtype
    y, order, p, _, _ = B.reference(d, top_k, norm)
    a = a_parts(R.normalized(d, norm, 1e-5), dtype)
    if lost_k:
        a[:, -1] = 0
    out = torch.zeros_like(y)
    for e in order.unique().tolist():
        m, s = (order == e).nonzero(as_tuple=True)
        gate, up = (a[m] @ d[n][e].double().t() for n in ("Wg", "Wu"))
        h = h_parts(p[m, s][:, None] * gate * torch.sigmoid(gate) * up, dtype)
        if lost_f:
            h[:, -1] = 0
        out[m] += h @ d["Wd"][e].double().t()
    return out.to(dtype).double()


def worst_of(d, top_k, norm):
    y, _, _, tol, _ = B.reference(d, top_k, norm)

    def worst(*parts, **lost):
        return ((layer(d, top_k, norm, *parts, **lost) - y).abs() / tol).max().item()

    return worst


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("norm", [0, 1, 2])
@pytest.mark.parametrize("M,K,F,E,top_k", B.CASES)
def test_a_lost_column_is_beyond_the_bound(M, K, F, E, top_k, norm, dtype):
    worst = worst_of(B.case(M, K, F, E, top_k, dtype, norm), top_k, norm)
    assert worst(two_parts, two_parts) <= 1
    assert worst(two_parts, two_parts, lost_k=True) > 1
    assert worst(two_parts, two_parts, lost_f=True) > 1


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("norm", [0, 2])
@pytest.mark.parametrize("M,K,F,E,top_k", B.CASES)
def test_a_lost_part_is_beyond_the_bound(M, K, F, E, top_k, norm, dtype):
    """In bf16 of a and of h, each by itself.  fp16's parts are 8 times as fine, which the sums' own errors hide in the
    wide cases."""
    worst = worst_of(B.sparse_case(M, K, F, E, top_k, dtype, norm), top_k, norm)
    assert worst(two_parts, two_parts) <= 1
    h = worst(two_parts, one_part)
    a = worst(one_part, two_parts) if norm else h      # (without a norm a is x, which one part holds)
    if dtype is BF16:
        assert min(a, h) > 1.2
    elif max(K, F) <= 256:
        assert max(a, h) > 1.2
