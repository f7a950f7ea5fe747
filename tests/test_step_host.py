"""Refusals of the rotated append, the paged attention and the experts, and
their workspaces' sizes: no GPU is needed, no address is dereferenced."""
import ctypes

import pytest
import torch

import normalization_gemm_row_gb300 as pkg
from normalization_gemm_row_gb300 import binding as B

A, OTHER, WS = 0x10000, 0x20000, 0x100000      # fake addresses
NULL, SHAPE, ALIGN, DTYPE, WORKSPACE, ARCH, CUDA, ARG = -1, -2, -3, -4, -5, -6, -7, -9


@pytest.fixture(scope="module", autouse=True)
def _lib():
    pkg.build()


def passes(rc):
    """Nothing refused: the call gets as far as the device (which this test must not reach)."""
    return rc in (ARCH, CUDA)


host_only = pytest.mark.skipif(torch.cuda.is_available(), reason="fake addresses must not reach a device")


def cache(**kw):
    f = dict(k=A, v=OTHER, pages=10, page_size=16, k_page_stride=16 * 2 * 64, k_token_stride=2 * 64, k_head_stride=64,
             v_page_stride=16 * 2 * 64, v_token_stride=2 * 64, v_head_stride=64, table=A, table_rows=4, table_pages=5, table_stride=5)
    f.update(kw)
    return B.KvCache(**f)


def append(c="default", **kw):
    f = dict(q=A, q_token=512, q_head=64, k=A, k_token=128, k_head=64, v=A, v_token=128, v_head=64,
             cache=cache() if c == "default" else c, positions=A, rows=None, inv_freq=A, rot=64, interleaved=0, T=4, H=8, G=2, D=64,
             dtype=0, q_out=OTHER, q_out_token=512, q_out_head=64, ws=None, ws_bytes=0, stream=None)
    f.update(kw)
    return B.ngr_fused_rope_append_kv(*f.values())


def attend(c="default", **kw):
    f = dict(q=A, q_row=512, q_head=64, cache=cache() if c == "default" else c, lengths=A, scale=0.1, window=0, B=4, H=8, G=2, D=64,
             dtype=0, out=A, lse=None, ws=WS, ws_bytes=1 << 30, stream=None)
    f.update(kw)
    return B.ngr_fused_paged_attention(*f.values())


def moe(**kw):
    f = dict(norm=2, x=A, gamma=A, beta=None, Wr=A, Wg=A, Wu=A, Wd=A, eps=1e-5, top_k=2, renormalize=1, M=4, K=64, F=96, E=8, dtype=0,
             y=A, experts=None, weights=None, ws=WS, ws_bytes=1 << 30, stream=None)
    f.update(kw)
    return B.ngr_fused_moe_swiglu(*f.values())


@pytest.mark.parametrize("rc,kw", [
    (DTYPE, dict(dtype=2)), (SHAPE, dict(T=-1)), (SHAPE, dict(G=0)), (SHAPE, dict(D=0)), (SHAPE, dict(D=257)), (SHAPE, dict(H=0)),
    (ARG, dict(rot=-2)), (ARG, dict(rot=7)), (ARG, dict(rot=66)), (NULL, dict(k=None)), (NULL, dict(v=None)), (NULL, dict(positions=None)),
    (NULL, dict(inv_freq=None)), (NULL, dict(q_out=None)), (NULL, dict(c=None)), (ALIGN, dict(k=A + 1)), (ALIGN, dict(q=A + 1)),
    (ALIGN, dict(q_out=A + 1)), (ALIGN, dict(positions=A + 2)), (ALIGN, dict(rows=A + 2)), (ALIGN, dict(inv_freq=A + 2)),
    (SHAPE, dict(T=5)),                                             # more tokens than rows of the table, and no rows given
    (ARG, dict(k_token=-128)), (ARG, dict(q_out_token=0)), (ARG, dict(q_out_head=32)), (ARG, dict(q_out=A, q_out_head=128)),
    (WORKSPACE, dict(ws=WS, ws_bytes=255)), (ALIGN, dict(ws=WS + 128, ws_bytes=256))])
def test_append_refuses(rc, kw):
    assert append(**kw) == rc


@pytest.mark.parametrize("rc,kw", [
    (NULL, dict(k=None)), (NULL, dict(v=None)), (NULL, dict(table=None)), (SHAPE, dict(pages=0)), (SHAPE, dict(page_size=0)),
    (SHAPE, dict(table_rows=0)), (SHAPE, dict(table_pages=0)), (ALIGN, dict(k=A + 1)), (ALIGN, dict(table=A + 2)),
    (ARG, dict(table_stride=4)), (ARG, dict(k_page_stride=-1)), (ARG, dict(v_head_stride=-64))])
def test_caches_are_refused(rc, kw):
    assert append(cache(**kw)) == rc
    assert attend(cache(**kw)) == rc


@pytest.mark.parametrize("kw", [dict(k_head_stride=0), dict(v_token_stride=0), dict(k_page_stride=0), dict(v_head_stride=32)])
def test_caches_whose_slots_overlap(kw):
    assert append(cache(**kw)) == ARG


@pytest.mark.parametrize("rc,kw", [
    (DTYPE, dict(dtype=-1)), (SHAPE, dict(B=-1)), (SHAPE, dict(H=7)), (SHAPE, dict(H=0)), (SHAPE, dict(G=0)), (SHAPE, dict(D=60)),
    (SHAPE, dict(D=264)), (SHAPE, dict(B=1 << 30)), (ARG, dict(scale=float("nan"))), (ARG, dict(scale=float("inf"))), (ARG, dict(window=-1)),
    (NULL, dict(q=None)), (NULL, dict(lengths=None)), (NULL, dict(out=None)), (NULL, dict(c=None)), (SHAPE, dict(B=5)),
    (ALIGN, dict(q=A + 2)), (ALIGN, dict(out=A + 8)), (ALIGN, dict(lengths=A + 1)), (ALIGN, dict(lse=A + 2)), (ALIGN, dict(q_head=66)),
    (WORKSPACE, dict(ws=None)), (WORKSPACE, dict(ws_bytes=255)), (ALIGN, dict(ws=WS + 16)), (ARG, dict(q_row=-512))])
def test_attention_refuses(rc, kw):
    assert attend(**kw) == rc


def test_attention_refuses_caches_off_the_boundary_and_beyond_64_gib():
    for kw in (dict(k=A + 2), dict(v=OTHER + 8), dict(k_token_stride=132), dict(v_page_stride=2050)):
        assert attend(cache(**kw)) == ALIGN
    assert attend(cache(pages=1 << 25, k_page_stride=1 << 10, v_page_stride=1 << 10)) == SHAPE      # 2^35 elements


@pytest.mark.parametrize("rc,kw", [
    (DTYPE, dict(dtype=5)), (ARG, dict(norm=3)), (ARG, dict(norm=-1)), (SHAPE, dict(M=33)), (SHAPE, dict(M=-1)), (SHAPE, dict(K=0)),
    (SHAPE, dict(F=0)), (SHAPE, dict(K=(1 << 20) + 1)), (SHAPE, dict(E=0)), (SHAPE, dict(E=1025)), (SHAPE, dict(top_k=0)), (SHAPE, dict(top_k=9)),
    (SHAPE, dict(top_k=33, E=64)), (ARG, dict(eps=-1.0)), (ARG, dict(eps=float("nan"))), (NULL, dict(x=None)), (NULL, dict(gamma=None)),
    (NULL, dict(norm=1)), (NULL, dict(Wr=None)), (NULL, dict(Wg=None)), (NULL, dict(Wu=None)), (NULL, dict(Wd=None)), (NULL, dict(y=None)),
    (ALIGN, dict(Wd=A + 1)), (ALIGN, dict(x=A + 1)), (ALIGN, dict(experts=A + 2)), (ALIGN, dict(weights=A + 1)),
    (WORKSPACE, dict(ws=None)), (WORKSPACE, dict(ws_bytes=1000)), (ALIGN, dict(ws=WS + 8))])
def test_experts_refuse(rc, kw):
    assert moe(**kw) == rc


def test_nothing_to_do():
    assert append(T=0, c=None) == 0 and attend(B=0, c=None, ws=None) == 0 and moe(M=0, x=None, ws=None) == 0


@host_only
def test_what_is_allowed():
    assert passes(append()) and passes(attend()) and passes(moe())
    assert passes(append(q=None, H=0, q_out=None)) and passes(append(rot=0, inv_freq=None)) and passes(append(T=9, rows=A))
    assert passes(append(q_out=A)) and passes(append(ws=WS, ws_bytes=256)) and passes(append(D=5, rot=4, q=A + 2, k_token=13))
    # strides of dimensions with one entry mean nothing
    assert passes(append(cache(pages=1, k_page_stride=-7), T=1, q_token=-3, q_out_token=0))
    assert passes(attend(B=1, q_row=3)) and passes(attend(cache(pages=1, k_page_stride=3)))
    assert passes(moe(norm=0, gamma=None, eps=-1.0)) and passes(moe(norm=1, beta=A)) and passes(moe(M=32, K=7, F=9, E=1024, top_k=32, x=A + 2))


def test_workspace_sizes():
    size = B.ngr_paged_attention_workspace_bytes
    assert size(4, 8, 2, 64, 80, 0) == 256                         # a CTA an item
    large = size(1, 64, 8, 128, 131072, 0)
    assert large > 1 << 20 and size(1, 64, 8, 128, 1 << 40, 0) == large and size(64, 64, 8, 128, 8192, 0) > 1 << 20
    assert size(1, 64, 8, 128, 131072, 1024) == 256                # a window is as short a context
    for bad in ((-1, 8, 2, 64, 80, 0), (4, 7, 2, 64, 80, 0), (4, 8, 2, 60, 80, 0), (4, 8, 2, 64, 0, 0), (4, 8, 2, 64, 80, -1)):
        assert size(*bad) == 0
    size = B.ngr_moe_swiglu_workspace_bytes
    assert size(1, 64, 96, 8, 2) > 0 and size(32, 4096, 14336, 8, 2) > size(1, 4096, 14336, 8, 2)
    for bad in ((33, 64, 96, 8, 2), (1, 0, 96, 8, 2), (1, 64, 96, 8, 9), (1, 64, 96, 1025, 2)):
        assert size(*bad) == 0
    assert ctypes.sizeof(B.KvCache) == 14 * 8


def test_helpers_refuse_on_the_cpu():
    t = torch.zeros((2, 4, 8), dtype=torch.float16)
    kv = torch.zeros((2, 4, 2, 8), dtype=torch.float16)
    table, pos = torch.zeros((2, 1), dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        pkg.fused_rope_append_kv(t, t[:, :2], t[:, :2], kv, kv, table, pos)
    with pytest.raises(ValueError, match="CUDA"):
        pkg.fused_paged_attention(t, kv, kv, table, pos)
    with pytest.raises(TypeError, match="float16 or bfloat16"):
        pkg.fused_paged_attention(t.float(), kv, kv, table, pos)
    with pytest.raises(TypeError, match="dtype"):
        pkg.fused_paged_attention(t, kv.bfloat16(), kv, table, pos)
    with pytest.raises(TypeError, match="int32"):
        pkg.fused_paged_attention(t, kv, kv, table.long(), pos)
    with pytest.raises(ValueError, match="caches"):
        pkg.fused_paged_attention(t, kv, kv[:1], table, pos)
    with pytest.raises(ValueError, match="caches"):
        pkg.fused_rope_append_kv(t, t, t, kv[0], kv[0], table, pos)
    with pytest.raises(ValueError, match="Wr must"):
        pkg.fused_moe_swiglu(t, kv[0, 0], kv[0], kv[0], kv[0], 1)
    w = torch.zeros((3, 5, 8), dtype=torch.float16)
    with pytest.raises(ValueError, match="gamma"):
        pkg.fused_moe_swiglu(t, torch.zeros((3, 8), dtype=torch.float16), w, w, w.transpose(1, 2).contiguous(), 1, norm=2,
                             gamma=torch.zeros(7, dtype=torch.float16))
    with pytest.raises(ValueError, match="CUDA"):
        pkg.fused_moe_swiglu(t, torch.zeros((3, 8), dtype=torch.float16), w, w, w.transpose(1, 2).contiguous(), 1)


@pytest.mark.parametrize("H,G,D", [(64, 8, 128), (4, 1, 64), (40, 2, 256), (12, 12, 80)])
@pytest.mark.parametrize("capacity", [16, 1000, 2048, 5000, 40000])
def test_a_workspace_is_enough_for_smaller_batches_and_tables(H, G, D, capacity):
    size = B.ngr_paged_attention_workspace_bytes
    of_batches = [size(n, H, G, D, capacity, 0) for n in range(1, 200)]
    assert of_batches == sorted(of_batches)
    for n in (1, 7, 100):
        assert size(n, H, G, D, capacity, 0) <= size(n, H, G, D, 2 * capacity, 0)
        assert size(n, H, G, D, capacity, 500) <= size(n, H, G, D, capacity, 0)


@pytest.mark.parametrize("K,F,E,top_k", [(64, 96, 8, 2), (4096, 1536, 64, 6), (1000, 2001, 13, 3), (192, 4544, 4, 4)])
def test_experts_workspace_is_enough_for_fewer_tokens(K, F, E, top_k):
    sizes = [B.ngr_moe_swiglu_workspace_bytes(m, K, F, E, top_k) for m in range(1, 33)]
    assert sizes == sorted(sizes)


@host_only
def test_query_heads_of_a_key_head():
    wide = cache(k_token_stride=64, k_head_stride=64, v_token_stride=64, v_head_stride=64)
    assert attend(wide, H=9729, G=1, q_row=9729 * 64) == SHAPE
    assert passes(attend(wide, H=9728, G=1, q_row=9728 * 64))
