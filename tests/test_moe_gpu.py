"""The mixture-of-experts layer for a few tokens against its formula in
float64: routing exactly, the output within its roundings."""
import pytest
import torch

import normalization_gemm_row_gb300 as ngr
import moe_reference as R

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _built():
    ngr.build()
    torch.cuda.init()


def call(d, top_k, norm=2, **kw):
    c = {k: v.cuda() if v is not None else None for k, v in d.items()}
    return ngr.fused_moe_swiglu(c["x"], c["Wr"], c["Wg"], c["Wu"], c["Wd"], top_k, norm=norm, gamma=c["gamma"], beta=c["beta"],
                                return_routing=True, **kw)


def run(M, K, F, E, top_k, dtype, norm=2, renormalize=True, seed=0):
    d = R.separate(R.case(M, K, F, E, dtype, seed, norm), top_k, norm)
    return R.check(call(d, top_k, norm, renormalize=renormalize), R.reference(d, top_k, norm, renormalize=renormalize))


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("norm", [0, 1, 2])
@pytest.mark.parametrize("renormalize", [False, True])
def test_norms(norm, renormalize, dtype):
    run(5, 256, 192, 8, 2, dtype, norm, renormalize)


@pytest.mark.parametrize("M", [1, 2, 7, 8, 9, 15, 16, 17, 31, 32])
def test_tokens(M):
    run(M, 256, 320, 12, 3, BF16, seed=M)


@pytest.mark.parametrize("K,F", [(1, 1), (7, 9), (8, 8), (63, 65), (64, 64), (65, 63), (1000, 2001), (1001, 500), (4096, 128),
                                 (4100, 72), (128, 4097), (8200, 40)])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_widths(K, F, dtype):
    run(4, K, F, 5, 2, dtype, norm=2 if K > 1 else 0, seed=K + F)


@pytest.mark.parametrize("E,top_k", [(1, 1), (2, 2), (3, 1), (8, 8), (9, 4), (33, 5), (64, 6), (65, 32), (160, 8), (1024, 4), (1000, 32)])
def test_experts(E, top_k):
    run(6, 64, 40, E, top_k, F16, seed=E + top_k)


@pytest.mark.parametrize("M,E,top_k", [(12, 2, 1), (12, 2, 2), (24, 3, 2), (32, 1, 1), (32, 4, 4), (32, 5, 3), (17, 4, 2), (9, 1, 1)])
@pytest.mark.parametrize("K,F", [(128, 96), (61, 45), (64, 1000)])
def test_few_experts_of_many_tokens(M, E, top_k, K, F):
    """More tokens an expert than share one reading of its weights."""
    run(M, K, F, E, top_k, BF16, seed=M + E)


@pytest.mark.parametrize("K,F", [(16, 3000), (130, 2500), (3000, 16), (8, 9), (200, 4544)])
@pytest.mark.parametrize("M", [1, 19])
def test_long_thin_experts(M, K, F):
    """Units of one step, and units that many workers share."""
    run(M, K, F, 8, 4, F16, seed=K)


def test_everybody_chooses_the_same_and_everybody_apart():
    d = R.case(32, 128, 96, 40, BF16, seed=3, norm=0)
    d["Wr"].zero_()
    d["x"][:, 0] = 1.0
    d["Wr"][:, 0] = -torch.arange(40, dtype=torch.float32).to(BF16)      # expert 0 first, for all
    R.check(call(d, 2, norm=0), R.reference(d, 2, norm=0))
    d["x"][:, :64] = 0
    d["x"][torch.arange(32), torch.arange(32)] = 4.0
    d["Wr"].zero_()
    d["Wr"][torch.arange(32), torch.arange(32)] = 1.0                    # token m: expert m
    R.check(call(d, 1, norm=0), R.reference(d, 1, norm=0))


def test_ties_go_to_the_lowest_expert():
    d = R.case(3, 64, 32, 70, F16, seed=4, norm=0)
    d["Wr"].zero_()
    y, experts, weights = call(d, 5, norm=0)
    assert (experts.cpu() == torch.arange(5, dtype=torch.int32)).all()
    assert torch.allclose(weights.cpu(), torch.full((3, 5), 0.2))
    d["Wr"][40:] = d["Wr"][40:] + 1.0
    d["x"] = d["x"].abs()
    _, experts, _ = call(d, 5, norm=0)
    assert (experts.cpu() == torch.arange(40, 45, dtype=torch.int32)).all()


def test_tokens_that_are_not_finite_stay_apart():
    d = R.separate(R.case(10, 128, 96, 12, BF16, seed=5), 3)
    want = R.reference(d, 3)
    bad = {2: float("nan"), 5: float("inf"), 9: -float("inf")}
    for m, v in bad.items():
        d["x"][m, 7] = v
    y, experts, weights = (t.cpu() for t in call(d, 3))
    keep = torch.tensor([m not in bad for m in range(10)])
    assert torch.isnan(y[~keep]).all() and torch.isnan(weights[~keep]).all()
    assert ((experts >= 0) & (experts < 12)).all()
    R.check((y[keep], experts[keep], weights[keep]), tuple(t[keep] for t in want))


def test_weights_of_experts_that_nobody_chooses_are_not_read():
    d = R.separate(R.case(2, 128, 96, 12, F16, seed=6), 2)
    want = R.reference(d, 2)
    idle = [e for e in range(12) if e not in want[1].unique().tolist()]
    for n in ("Wg", "Wu", "Wd"):
        d[n][idle] = float("nan")
    R.check(call(d, 2), want)


def test_addresses_off_the_boundary():
    """Weights, rows and outputs that start at any element."""
    d = R.separate(R.case(3, 128, 64, 6, BF16, seed=7), 2)
    want = R.reference(d, 2)
    for off in (1, 3, 8):
        c = {}
        for k, v in d.items():
            if v is not None:
                flat = torch.zeros(v.numel() + off, dtype=v.dtype, device="cuda")
                flat[off:] = v.cuda().flatten()
                c[k] = flat[off:].view(v.shape)
        got = ngr.fused_moe_swiglu(c["x"], c["Wr"], c["Wg"], c["Wu"], c["Wd"], 2, norm=2, gamma=c["gamma"], return_routing=True,
                                   out=c["x"])
        assert got[0] is c["x"]
        R.check(got, want, f"offset {off}")


def test_shapes_and_repeats():
    d = R.separate(R.case(6, 128, 64, 6, F16, seed=8), 2)
    d2 = {k: v.cuda() if v is not None else None for k, v in d.items()}
    x = d2["x"].view(2, 3, 128)
    y, e, w = ngr.fused_moe_swiglu(x, d2["Wr"], d2["Wg"], d2["Wu"], d2["Wd"], 2, norm=2, gamma=d2["gamma"], return_routing=True)
    assert y.shape == (2, 3, 128) and e.shape == (2, 3, 2) and w.shape == (2, 3, 2)
    again = ngr.fused_moe_swiglu(x, d2["Wr"], d2["Wg"], d2["Wu"], d2["Wd"], 2, norm=2, gamma=d2["gamma"])
    assert torch.equal(y, again)
    none = ngr.fused_moe_swiglu(x[:0], d2["Wr"], d2["Wg"], d2["Wu"], d2["Wd"], 2, norm=2, gamma=d2["gamma"])
    assert none.shape == (0, 3, 128)


@pytest.mark.parametrize("M,E,top_k", [(1, 3, 1), (2, 16, 4), (8, 16, 4), (29, 20, 5), (32, 24, 6)])
@pytest.mark.parametrize("F", [6000, 6001])
def test_rows_that_many_workers_share(M, E, top_k, F):
    """A few rows of down's result, each of them from thousands of steps."""
    run(M, 40, F, E, top_k, BF16, seed=M + F)
