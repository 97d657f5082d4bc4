"""The gradient of moe_product_fp8's rows with several weight matrices."""
import numpy as np
import pytest
import torch

import combine_topk_ids_gb300 as moe
from oracle import fp8 as ofp8
from oracle.block import EPS32
from test_grouped_gpu import built, codes_of, draw_ids, f64, sort_picks, within  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,k,E,N,K", [(5, 2, 6, 384, 256), (70, 4, 8, 256, 640), (900, 2, 3, 512, 384), (60, 1, 3, 2048, 128)])
def test_gradient_of_the_rows_with_offsets(T, k, E, N, K):
    """d(a) of out[rows of e] = a b[e]^T: the product of out's gradient with each matrix's transposed codes and
    scales, by the same offsets; against the formula, and against differences of the product itself, which is
    linear in a."""
    offsets = sort_picks(draw_ids(T, k, E, 0.2, 3, skew=True), E)["offsets"]
    off, M = offsets.tolist(), T * k
    dy, sy = codes_of(M, N, block=1, seed=1)
    b, sb = codes_of(E, N, K, block=128, seed=2)
    bt, sbt = b.view(torch.uint8).transpose(1, 2).contiguous(), sb.transpose(1, 2).contiguous()
    da = torch.full((M, K), 7.0, device="cuda")
    moe.moe_product_fp8(dy, sy, bt, sbt, da, offsets=offsets)
    assert (da[off[-1]:] == 7).all()
    w = [ofp8.decode_e4m3(b[e].view(torch.uint8).cpu().numpy()) * np.repeat(np.repeat(f64(sb[e]), 128, 0), 128, 1) for e in range(E)]
    g = ofp8.decode_e4m3(dy.view(torch.uint8).cpu().numpy()) * np.repeat(f64(sy), 128, 1)
    size = np.zeros((M, K))
    for e in range(E):
        r = slice(off[e], off[e + 1])
        size[r] = np.abs(g[r]) @ np.abs(w[e])
        bound = (128 * 2.0 ** -23 + (N // 128 + 5) * EPS32) * size[r]
        within(f64(da[r]), g[r] @ w[e], bound + EPS32 * size[r], "da of expert %d" % e)
    # differences: a's code at one column of every row between 1 and -1 (0x38 and 0xb8), so that the
    # float64 sum of out * dy changes by twice the scale times da
    a, sa = codes_of(M, K, block=1, seed=5)
    a = a.view(torch.uint8)
    out, got = torch.zeros((M, N), device="cuda"), []
    for i in (0, K // 2 + 1, K - 1):
        sums = []
        for code in (0x38, 0xb8):
            c = a.clone()
            c[:, i] = code
            moe.moe_product_fp8(c, sa, b, sb, out, offsets=offsets)
            sums.append((f64(out) * g).sum(1))
        d = (sums[0] - sums[1]) / (2 * f64(sa)[:, i // 128])
        # each of out's two float32 values is off by at most chain * (|a| |b|^T), weighted with |dy|
        for e in range(E):
            r = slice(off[e], off[e + 1])
            va = np.abs(ofp8.decode_e4m3(a[r].cpu().numpy()))
            va[:, i] = np.maximum(va[:, i], 1)
            chain = 128 * 2.0 ** -23 + (K // 128 + 6) * EPS32
            off_by = ((va * np.repeat(f64(sa[r]), 128, 1)) @ np.abs(w[e]).T * np.abs(g[r])).sum(1)
            near = chain * off_by / f64(sa[r])[:, i // 128] + (128 * 2.0 ** -23 + (N // 128 + 6) * EPS32) * size[r][:, i]
            within(d[r], f64(da[r])[:, i], near, "differences of expert %d, column %d" % (e, i))
        got.append(d)
    assert np.abs(np.stack(got)).max() > 0
