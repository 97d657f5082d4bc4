"""moe_product_fp8 by every kind of tile and every number of blocks that share one, against the oracle."""
import numpy as np
import pytest
import torch

import combine_topk_ids_gb300 as moe
from test_grouped_gpu import BF, F32, I32, built, check_product, codes_of, strided  # noqa: F401
from test_product_tiles import MANY, ONE

pytestmark = pytest.mark.gpu


def into_places(a, sa, b, sb, out, **kw):
    """The same product into rows that lie apart, on 16 bytes and off them, of rows that lie apart."""
    M, N = out.shape
    a = strided(a.view(torch.uint8), a.shape[1] + 16)
    for lead, off in ((16, 0), (3, 1)):
        room = torch.full((M * (N + lead) + off,), 7.0, dtype=out.dtype, device="cuda")
        part = room[off:].view(M, N + lead)
        moe.moe_product_fp8(a, sa, b, sb, part[:, :N], **kw)
        assert torch.equal(part[:, :N], out) and (part[:, N:] == 7).all() and (room[:off] == 7).all()


@pytest.mark.parametrize("M,N,K,rows,split", ONE)
@pytest.mark.parametrize("dtype", [BF, F32])
def test_one_matrix(M, N, K, rows, split, dtype):
    a, sa = codes_of(M, K, block=1, seed=1)
    b, sb = codes_of(N, K, block=128, seed=2)
    out, status = torch.full((M, N), float("nan"), dtype=dtype, device="cuda"), torch.zeros(1, dtype=I32, device="cuda")
    moe.moe_product_fp8(a, sa, b, sb, out, status=status)
    check_product(out, a, sa, b, sb)
    again = torch.empty_like(out)
    moe.moe_product_fp8(a, sa, b, sb, again, status=status)
    assert torch.equal(again, out)                       # equal inputs, equal bits
    into_places(a, sa, b, sb, out, status=status)
    assert status.item() == 0


def draw_offsets(M, G, seed):
    """Groups of all sizes, none among them, and a row behind the last one where there are several."""
    rng = np.random.default_rng(seed)
    off = np.sort(rng.integers(0, M + 1, G + 1))
    off[0], off[-1] = 0, M - (M > 4)
    off[G // 2] = off[G // 2 - 1]
    return off.clip(0, off[-1]).tolist()


@pytest.mark.parametrize("M,N,K,G,rows,split", MANY)
@pytest.mark.parametrize("dtype", [BF, F32])
def test_many(M, N, K, G, rows, split, dtype):
    off = draw_offsets(M, G, M + G)
    a, sa = codes_of(M, K, block=1, seed=1)
    a.view(torch.uint8)[off[-1]:] = 0x7f
    sa[off[-1]:] = float("nan")
    b, sb = codes_of(G, N, K, block=128, seed=2)
    out, status = torch.full((M, N), 7.0, dtype=dtype, device="cuda"), torch.zeros(1, dtype=I32, device="cuda")
    kw = dict(offsets=torch.tensor(off, dtype=I32, device="cuda"), status=status)
    moe.moe_product_fp8(a, sa, b, sb, out, **kw)
    for e in range(G):
        r = slice(off[e], off[e + 1])
        if r.start < r.stop:
            check_product(out[r], a[r], sa[r], b[e], sb[e], "expert %d" % e)
    assert (out[off[-1]:] == 7).all()
    again = torch.full_like(out, 7)
    moe.moe_product_fp8(a, sa, b, sb, again, **kw)
    assert torch.equal(again, out)
    into_places(a, sa, b, sb, out, **kw)
    # all rows in one group, the first or the last: clusters without a tile
    for one in (0, G - 1):
        kw["offsets"] = torch.tensor([0] * (one + 1) + [M] * (G - one), dtype=I32, device="cuda")
        moe.moe_product_fp8(a, sa, b, sb, again, **kw)
        r = slice(0, off[-1])
        check_product(again[r], a[r], sa[r], b[one], sb[one], "expert %d alone" % one)
    assert status.item() == 0
