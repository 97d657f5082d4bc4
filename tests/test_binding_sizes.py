"""Sizes that the C structs' 32-bit fields do not hold: refused by the binding with MOE_ERR_LIMIT, where ctypes would
cut them off and the call would take a part of its tensors for the whole.  (Tensors without memory.)"""
import os

import pytest
import torch

import combine_topk_ids_gb300 as moe

BF, F32, I32, U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8
BIG = (1 << 32) + 128      # taken for 128


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not os.path.exists(moe.LIB_PATH):
        moe.build()
    return moe.lib()


def m(*shape, dtype=BF):
    return torch.empty(shape, dtype=dtype, device="meta")


def limit(call, *args, **kw):
    with pytest.raises(moe.MoeError) as e:
        call(*args, **kw)
    assert e.value.code == -13, e.value


@pytest.mark.parametrize("T,k,E", [(BIG, 1, 8), (1 << 31, 1, 8), (4, BIG, 8), (4, 1, BIG)])
def test_sort_picks(T, k, E):
    limit(moe.moe_sort_picks_workspace_size, T, k, E)
    limit(moe.moe_sort_picks, m(T, k, dtype=torch.int64), E, m(E + 1, dtype=I32), m(T, k, dtype=I32), m(1 << 20, dtype=U8))


@pytest.mark.parametrize("T,k,R,H", [(BIG, 1, 8, 1), (2, BIG, 8, 4), (2, 2, BIG, 4), (1, 1, 1, BIG), (1, 1, 1 << 31, 2)])
def test_rows(T, k, R, H):
    position, w = m(T, k, dtype=I32), m(T, k, dtype=F32)
    limit(moe.moe_sort_rows, m(T, H), position, m(R, H))
    limit(moe.moe_sort_rows_backward, m(R, H), position, m(T, H))
    limit(moe.moe_unsort_rows, m(R, H), w, position, m(T, H))
    limit(moe.moe_unsort_rows_backward, m(T, H), m(R, H), w, position, m(R, H), w)
    limit(moe.moe_unsort_rows_backward, m(T, H), None, w, position, m(R, H), None)


@pytest.mark.parametrize("R,C", [(BIG, 128), (1, BIG)])
def test_quantize(R, C):
    limit(moe.moe_quantize_fp8, m(R, C), m(R, C, dtype=U8), m(R, C // 128, dtype=F32))
    limit(moe.moe_quantize_fp8, m(R, 2, 128), m(R, 2, 128, dtype=U8), m(R, 1, 1, dtype=F32), block_rows=128) if R > 1 else None
    limit(moe.moe_swiglu_fp8, m(R, 2 * C), m(R, C, dtype=U8), m(R, C // 128, dtype=F32))


@pytest.mark.parametrize("M,N,K,G", [(BIG, 128, 128, 0), (2, BIG, 128, 0), (2, 128, BIG, 0), (2, 128, 128, BIG)])
def test_product(M, N, K, G):
    lead = (G,) if G else ()
    limit(moe.moe_product_fp8, m(M, K, dtype=U8), m(M, K // 128, dtype=F32), m(*lead, N, K, dtype=U8),
          m(*lead, -(-N // 128), K // 128, dtype=F32), m(M, N), offsets=m(G + 1, dtype=I32) if G else None)


@pytest.mark.parametrize("T,H", [(BIG, 4), (1, BIG)])
def test_norm_and_router(T, H):
    x, w, rstd = m(T, H), m(H), m(T, dtype=F32)
    limit(moe.moe_add_rmsnorm, x, None, w, 1e-6, out=m(T, H))
    limit(moe.moe_add_rmsnorm_workspace_size, T, H)
    limit(moe.moe_add_rmsnorm_backward, x, x, w, rstd, m(T, H), m(H, dtype=F32), m(64, dtype=U8))
    if T > 1:
        router = moe.make_router(8, 2)
        ids, weights = m(T, 2, dtype=I32), m(T, 2, dtype=F32)
        limit(moe.moe_route_topk, router, m(T, 8), None, ids, weights)
        limit(moe.moe_route_topk_backward, router, m(T, 8), ids, weights, m(T, 8))
