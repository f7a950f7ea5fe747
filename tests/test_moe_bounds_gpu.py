"""The mixture-of-experts layer against the bound of moe_bounds.py: what one
rounding of a or h, a lost second part or a lost column would exceed."""
import pytest
import torch

import normalization_gemm_row_gb300 as ngr
import moe_bounds as B
import moe_reference as R

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _built():
    ngr.build()
    torch.cuda.init()


def check(d, top_k, norm, what=""):
    c = {k: v.cuda() if v is not None else None for k, v in d.items()}
    got = ngr.fused_moe_swiglu(c["x"], c["Wr"], c["Wg"], c["Wu"], c["Wd"], top_k, norm=norm, gamma=c["gamma"], beta=c["beta"],
                               return_routing=True)
    return R.check(got, B.reference(d, top_k, norm), what)


def scaled(d, **by):
    return {k: (v.double() * by.get(k, 1.0)).to(v.dtype) if v is not None else None for k, v in d.items()}


@pytest.mark.parametrize("M,K,F,E,top_k", [(1, 64, 48, 4, 2), (6, 256, 200, 8, 3), (32, 61, 45, 4, 2)])
def test_fp16_values_beyond_the_ends_of_its_range(M, K, F, E, top_k):
    """h of 1e5 to 1e7, of 1e-9 to 1e-5, and normalized rows of 1e-5."""
    for norm, by in ((0, {"Wg": 1500.0, "Wu": 1500.0, "Wd": 1e-3}), (0, {"Wg": 2e-3, "Wu": 1e-3, "Wd": 60.0}),
                     (2, {"gamma": 1e-5, "Wg": 100.0, "Wu": 100.0, "Wd": 60.0})):
        d = scaled(R.separate(R.case(M, K, F, E, F16, seed=M, norm=norm), top_k, norm), **by)
        if "gamma" in by:
            d["Wr"] = (d["Wr"].double() * 500).to(F16)
            d = R.separate(d, top_k, norm)
        check(d, top_k, norm, str(by))


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("norm", [0, 1, 2])
@pytest.mark.parametrize("M,K,F,E,top_k", B.CASES)
def test_every_column_counts(M, K, F, E, top_k, norm, dtype):
    check(B.case(M, K, F, E, top_k, dtype, norm), top_k, norm)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("norm", [0, 2])
@pytest.mark.parametrize("M,K,F,E,top_k", B.CASES)
def test_both_parts_count(M, K, F, E, top_k, norm, dtype):
    check(B.sparse_case(M, K, F, E, top_k, dtype, norm), top_k, norm)
