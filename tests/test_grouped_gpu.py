"""The operators on expert-grouped rows on the GPU, through the public entry points, against the
float64 oracle, at the sizes, strides and masks where they can go wrong."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import combine_topk_ids_gb300 as moe
from oracle import fp8 as ofp8
from oracle import grouped as og
from oracle.block import BF16, E4M3, EPS32

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
pytestmark = pytest.mark.gpu
BF, F32, I32, F8 = torch.bfloat16, torch.float32, torch.int32, torch.float8_e4m3fn
HALF = {BF: BF16, F32: EPS32}


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    if not os.path.exists(moe.LIB_PATH):
        moe.build()


def f64(t):
    return t.detach().cpu().double().numpy()


def rnd(*shape, dtype=BF, scale=1.0, seed=0):
    g = torch.Generator().manual_seed(seed + 1000 * len(shape) + sum(shape))
    return (torch.randn(shape, generator=g) * scale).to(dtype).cuda()


def strided(t, lead, off=0):
    """The same matrix with rows `lead` elements apart, `off` elements into its storage."""
    buf = torch.full((t.shape[0] * lead + off,), 7.0, device=t.device).to(t.dtype)
    v = buf[off:].view(t.shape[0], lead)[:, :t.shape[1]]
    v.copy_(t)
    return v


def within(got, ref, bound, what):
    d = np.abs(got - ref)
    bad = ~(d <= bound)
    assert not bad.any(), "%s: %d of %d outside; worst %.3g at %s" % (
        what, bad.sum(), bad.size, d[bad].max(), np.argwhere(bad)[0])


def draw_ids(T, k, E, drop=0.0, seed=0, skew=False):
    rng = np.random.default_rng(seed)
    ids = rng.integers(0, E, (T, k)) if not skew else np.minimum(rng.geometric(0.4, (T, k)) - 1, E - 1)
    ids[rng.random((T, k)) < drop] = -1
    return ids


def sort_picks(ids, E, dtype=torch.int64, **kw):
    T, k = ids.shape
    r = {"offsets": torch.full((E + 1,), -7, dtype=I32, device="cuda"),
         "position": torch.full((T, k), -7, dtype=I32, device="cuda"),
         "source": torch.full((T * k,), -7, dtype=I32, device="cuda"),
         "status": torch.full((1,), -7, dtype=I32, device="cuda")}
    work = torch.empty(moe.moe_sort_picks_workspace_size(T, k, E), dtype=torch.uint8, device="cuda").fill_(255)
    moe.moe_sort_picks(torch.tensor(ids).to(dtype).cuda(), E, r["offsets"], r["position"], work, source=r["source"],
                       status=r["status"], **kw)
    return r


def check_order(r, ids, E):
    offsets, position, source = og.order(ids, E)
    np.testing.assert_array_equal(r["offsets"].cpu().numpy(), offsets)
    np.testing.assert_array_equal(r["position"].cpu().numpy(), position)
    np.testing.assert_array_equal(r["source"].cpu().numpy(), source)
    assert r["status"].item() == (1 if ((ids < -1) | (ids >= E)).any() else 0)


# ---- order ---------------------------------------------------------------------------------------

@pytest.mark.parametrize("T,k,E", [(0, 2, 5), (1, 1, 1), (1, 32, 4), (3, 2, 8), (64, 8, 256), (31, 7, 60), (512, 8, 64),
                                   (513, 8, 64), (1000, 8, 2048), (511, 8, 2048), (3000, 5, 1025), (9000, 4, 128),
                                   (16381, 4, 128), (33000, 8, 33), (4097, 1, 3)])
@pytest.mark.parametrize("drop,skew", [(0.0, False), (0.3, True)])
def test_order(T, k, E, drop, skew):
    ids = draw_ids(T, k, E, drop, T + E, skew)
    check_order(sort_picks(ids, E), ids, E)
    check_order(sort_picks(ids, E, torch.int32), ids, E)


@pytest.mark.parametrize("T,k,E", [(40, 4, 8), (5000, 4, 8)])
def test_order_of_odd_batches(T, k, E):
    """Nothing left, one expert alone, ids that are none (one only, in one block), the same twice."""
    for ids in (np.full((T, k), -1), np.full((T, k), E - 1), np.zeros((T, k), np.int64)):
        check_order(sort_picks(ids, E), ids, E)
    ids = draw_ids(T, k, E, 0.1)
    for bad in (E, -2, 1 << 40, -(1 << 40)):
        one = ids.copy()
        one[T - 1, k - 1] = bad
        check_order(sort_picks(one, E), one, E)
    g, work = moe.moe_sort_picks, torch.empty(moe.moe_sort_picks_workspace_size(T, k, E), dtype=torch.uint8, device="cuda")
    offsets, position = torch.empty(E + 1, dtype=I32, device="cuda"), torch.empty((T, k), dtype=I32, device="cuda")
    g(torch.tensor(ids).cuda(), E, offsets, position, work)     # without source and status
    check = og.order(ids, E)
    np.testing.assert_array_equal(offsets.cpu().numpy(), check[0])
    np.testing.assert_array_equal(position.cpu().numpy(), check[1])


# ---- rows ----------------------------------------------------------------------------------------

ROWS = [(1, 1, 1), (1, 8, 7168), (3, 2, 7), (5, 4, 2047), (7, 32, 130), (9, 3, 128), (33, 6, 513), (130, 8, 256),
        (4, 2, 65536), (3, 9, 16385), (600, 2, 64)]


def plan(T, k, seed=0, drop=0.2):
    ids = draw_ids(T, k, 4, drop if T > 1 else 0.0, seed)
    if T > 2:
        ids[1] = -1           # a token without picks
    return ids, sort_picks(ids, 4)["position"]


@pytest.mark.parametrize("T,k,H", ROWS)
@pytest.mark.parametrize("dtype", [BF, F32, F8])
@pytest.mark.parametrize("lead,off", [(0, 0), (1, 1), (8, 0), (8, 3)])
def test_sort_rows(T, k, H, dtype, lead, off):
    if dtype == F8 and (H % 128 or lead):
        return
    ids, position = plan(T, k)
    x = rnd(T, H, dtype=F32).to(dtype)
    R = T * k + 3
    rows = rnd(R, H, dtype=F32, seed=5).to(dtype)
    kw = {}
    if dtype == F8:
        kw = dict(x_scales=rnd(T, H // 128, dtype=F32), rows_scales=rnd(R, H // 128, dtype=F32, seed=1))
        want_scales = og.sort_rows(f64(kw["x_scales"]), position.cpu().numpy(), f64(kw["rows_scales"]))
    elif lead:
        x, rows = strided(x, H + lead, off), strided(rows, H + 2 * lead, off)
    want = og.sort_rows(f64(x.float()), position.cpu().numpy(), f64(rows.float()))
    moe.moe_sort_rows(x, position, rows, **kw)
    np.testing.assert_array_equal(f64(rows.float()), want)      # rows of no pick among them
    if dtype == F8:
        np.testing.assert_array_equal(f64(kw["rows_scales"]), want_scales)


@pytest.mark.parametrize("T,k,H", ROWS)
@pytest.mark.parametrize("rt,ot", [(BF, BF), (BF, F32), (F32, BF), (F32, F32)])
@pytest.mark.parametrize("lead,off", [(0, 0), (1, 1), (8, 4)])
def test_unsort_rows_and_gradients(T, k, H, rt, ot, lead, off):
    ids, position = plan(T, k, 1)
    pos = position.cpu().numpy()
    R = T * k
    rows, dout, w = rnd(R, H, dtype=rt), rnd(T, H, dtype=ot, seed=1), rnd(T, k, dtype=F32, seed=2)
    w[position < 0] = float("nan")                 # a masked pick's weight is not read
    rows[int((pos >= 0).sum()):] = float("nan")    # nor are rows that no pick has
    out = torch.full((T, H), 3.0, dtype=ot, device="cuda")
    drows = rnd(R, H, dtype=rt, seed=4)
    if lead:
        rows, dout, out, drows = (strided(t, H + n * lead, off) for n, t in ((1, rows), (2, dout), (3, out), (1, drows)))
    r64, d64, w64 = f64(rows), f64(dout), f64(w)
    for weights in (w, None):
        v = None if weights is None else w64
        moe.moe_unsort_rows(rows, weights, position, out)
        ref, bound = og.unsort_rows(r64, v, pos)
        within(f64(out), ref, bound + HALF[ot] * (np.abs(ref) + bound), "out")
        before = f64(drows)
        dw = torch.full((T, k), 5.0, device="cuda")
        moe.moe_unsort_rows_backward(dout, rows, weights, position, drows, dw)
        g, gw, bw = og.unsort_rows_backward(d64, r64, v, pos, before)
        within(f64(drows), g, (HALF[rt] + EPS32) * np.abs(g), "drows")
        within(f64(dw), gw, bw, "dweights")
        # one at a time: the same bits
        only = torch.empty_like(dw)
        moe.moe_unsort_rows_backward(dout, rows, weights, position, None, only)
        assert torch.equal(only, dw)
        again = torch.empty_like(drows)
        again.copy_(torch.tensor(before))
        moe.moe_unsort_rows_backward(dout, None, weights, position, again, None)
        assert torch.equal(again, drows)
    if rt == ot:
        dx = torch.empty_like(out)
        moe.moe_sort_rows_backward(rows, position, dx)
        assert torch.equal(dx, out)      # moe_unsort_rows without weights


def test_unsort_gradient_by_differences():
    T, k, H = 6, 3, 40
    ids, position = plan(T, k, 2)
    rows, dout, w = rnd(T * k, H, dtype=F32), rnd(T, H, dtype=F32, seed=1), rnd(T, k, dtype=F32, seed=2)
    drows, dw, out = torch.zeros_like(rows), torch.empty_like(w), torch.empty_like(dout)
    moe.moe_unsort_rows_backward(dout, rows, w, position, drows, dw)

    def loss():
        moe.moe_unsort_rows(rows, w, position, out)
        return (out.double() * dout.double()).sum().item()

    # linear in each: differences of size 1 are exact but for float32 sums of some 120 terms
    for v, g in ((rows, drows), (w, dw)):
        for i in [(0, 0), (T - 1, k - 1), (2, 1), (3, 2)]:
            keep = v[i].item()
            v[i] = keep + 1
            up = loss()
            v[i] = keep - 1
            down = loss()
            v[i] = keep
            assert abs((up - down) / 2 - g[i].item()) < 2e-4


def test_positions_outside_the_rows():
    """Positions that the matrix does not have take no part."""
    T, k, H = 5, 2, 256
    position = torch.tensor([[0, 9], [-1, 1], [10, 2], [1 << 30, -5], [3, 11]], dtype=I32, device="cuda")
    x, rows, w = rnd(T, H), rnd(10, H, seed=1), rnd(T, k, dtype=F32)
    want = og.sort_rows(f64(x), position.cpu().numpy(), f64(rows))
    moe.moe_sort_rows(x, position, rows)
    np.testing.assert_array_equal(f64(rows), want)
    out, drows, dw = torch.empty_like(x), torch.zeros_like(rows), torch.empty_like(w)
    moe.moe_unsort_rows(rows, w, position, out)
    ref, bound = og.unsort_rows(f64(rows), f64(w), position.cpu().numpy())
    within(f64(out), ref, bound + HALF[BF] * (np.abs(ref) + bound), "out")
    moe.moe_unsort_rows_backward(x, rows, w, position, drows, dw)
    g, gw, bw = og.unsort_rows_backward(f64(x), f64(rows), f64(w), position.cpu().numpy(), np.zeros((10, H)))
    within(f64(drows), g, (HALF[BF] + EPS32) * np.abs(g), "drows")
    within(f64(dw), gw, bw, "dweights")


def test_rows_empty():
    position = torch.empty((0, 2), dtype=I32, device="cuda")
    x, rows = torch.empty((0, 64), dtype=BF, device="cuda"), rnd(4, 64)
    keep = rows.clone()
    moe.moe_sort_rows(x, position, rows)
    moe.moe_unsort_rows(rows, None, position, x)
    moe.moe_unsort_rows_backward(x, rows, None, position, rows, torch.empty((0, 2), device="cuda"))
    assert torch.equal(rows, keep)
    position = torch.full((3, 2), -1, dtype=I32, device="cuda")
    out, none, dw = rnd(3, 64), torch.empty((0, 64), dtype=BF, device="cuda"), torch.ones((3, 2), device="cuda")
    moe.moe_sort_rows(out, position, none)
    moe.moe_unsort_rows_backward(out, none, None, position, none, dw)
    assert not dw.any()
    moe.moe_unsort_rows(none, None, position, out)      # rows that there are none of: zeros
    assert not out.any()


# ---- quantisation --------------------------------------------------------------------------------

@pytest.mark.parametrize("R,C", [(1, 128), (5, 256), (3, 7168), (130, 384), (257, 640), (64, 4096)])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("lead,off", [(0, 0), (1, 1), (8, 0)])
def test_quantize(R, C, dtype, lead, off):
    x = rnd(R, C, dtype=dtype) * torch.logspace(-40, 6, R, device="cuda")[:, None].to(dtype)
    x[0, :128] = 0
    if R > 2:
        x[2, 5], x[2, 6] = 448.0, -1e-3
    if lead:
        x = strided(x, C + lead, off)
    codes, scales = torch.empty((R, C), dtype=F8, device="cuda"), torch.empty((R, C // 128), device="cuda")
    moe.moe_quantize_fp8(x, codes, scales)
    want, sc, _ = ofp8.quantize_rows(f64(x))
    np.testing.assert_array_equal(scales.cpu().numpy(), sc)
    np.testing.assert_array_equal(codes.view(torch.uint8).cpu().numpy(), want)
    bytes_, again = torch.empty((R, C), dtype=torch.uint8, device="cuda"), torch.full_like(scales, 3)
    live = torch.tensor([R // 2], dtype=I32, device="cuda")
    bytes_.fill_(9)
    moe.moe_quantize_fp8(x, bytes_, again, live_rows=live)
    n = R // 2
    np.testing.assert_array_equal(bytes_[:n].cpu().numpy(), want[:n])
    assert (bytes_[n:] == 9).all() and (again[n:] == 3).all()      # left as they were
    # 128 rows to a scale, the last block a short one
    RB = -(-R // 128)
    wide = torch.empty((RB, C // 128), device="cuda")
    moe.moe_quantize_fp8(x, bytes_, wide, block_rows=128)
    v = f64(x).astype(np.float32)
    for b in range(RB):
        part = v[128 * b:128 * b + 128].reshape(-1, C // 128, 128)
        a = np.maximum(np.abs(part).max((0, 2)), np.float32(2.0 ** -100))
        np.testing.assert_array_equal(wide[b].cpu().numpy(), a / np.float32(448))
        quo = part * (np.float32(448) / a)[:, None]
        np.testing.assert_array_equal(bytes_[128 * b:128 * b + 128].cpu().numpy(), ofp8.round_e4m3(quo.astype(np.float64)).reshape(-1, C))


def test_quantize_matrices():
    """Several matrices, none of whose blocks reaches into the next."""
    x = rnd(3, 2, 200, 256)
    codes, scales = torch.empty(x.shape, dtype=F8, device="cuda"), torch.empty((3, 2, 2, 2), device="cuda")
    moe.moe_quantize_fp8(x, codes, scales, block_rows=128)
    for i in range(3):
        for j in range(2):
            c, s = torch.empty((200, 256), dtype=F8, device="cuda"), torch.empty((2, 2), device="cuda")
            moe.moe_quantize_fp8(x[i, j], c, s, block_rows=128)
            assert torch.equal(c.view(torch.uint8), codes[i, j].view(torch.uint8)) and torch.equal(s, scales[i, j])


def test_quantize_what_is_no_number():
    x = rnd(3, 256, dtype=F32)
    x[0, 3], x[1, 200], x[2, 7] = float("nan"), float("inf"), -float("inf")
    for block in (1, 128):
        codes = torch.empty((3, 256), dtype=F8, device="cuda")
        scales = torch.empty((3 if block == 1 else 1, 2), device="cuda")
        moe.moe_quantize_fp8(x, codes, scales, block_rows=block)
        v = codes.float() * scales.repeat_interleave(block, 0)[:3].repeat_interleave(128, 1)
        if block == 1:
            assert v[0].isnan().nonzero().flatten().tolist() == [3]
            assert v[1, :128].isfinite().all() and v[1, 128:].isnan().all()
            assert v[2, :128].isnan().all() and v[2, 128:].isfinite().all()
        else:
            assert v.isnan().all()
    g = torch.zeros((1, 512), device="cuda")
    g[0, :256] = torch.linspace(-200, 200, 256, device="cuda")
    g[0, 0], g[0, 255] = -1e30, 1e30
    g[0, 256:] = 1
    codes, scales = torch.empty((1, 256), dtype=F8, device="cuda"), torch.empty((1, 2), device="cuda")
    moe.moe_swiglu_fp8(g, codes, scales)
    assert (codes.float().isfinite()).all() and scales.isfinite().all()


@pytest.mark.parametrize("R,C", [(1, 128), (3, 2048), (130, 384), (40, 1408)])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("lead", [0, 1, 8])
def test_swiglu(R, C, dtype, lead):
    x = rnd(R, 2 * C, dtype=dtype) * torch.logspace(-3, 1.5, R, device="cuda")[:, None].to(dtype)
    if lead:
        x = strided(x, 2 * C + lead)
    codes, scales = torch.empty((R, C), dtype=F8, device="cuda"), torch.empty((R, C // 128), device="cuda")
    moe.moe_swiglu_fp8(x, codes, scales)
    v, rel = og.swiglu(f64(x))
    top = np.maximum(np.abs(v).reshape(R, -1, 128).max(2), 2.0 ** -100)
    within(f64(scales), top / 448, (rel + EPS32) * top / 448, "scales")
    sc = np.repeat(f64(scales), 128, 1)
    # half a code in the normal range, half the smallest step (2^-10) below it
    within(f64(codes.float()) * sc, v, (E4M3 + 2 * rel) * np.abs(v) + 2.0 ** -10 * 1.001 * sc, "codes")


# ---- product -------------------------------------------------------------------------------------

def codes_of(*shape, block, seed):
    """Codes and scales of random rows of different size (block 1) or of weights (128)."""
    x = rnd(*shape, dtype=F32, seed=seed)
    if block == 1:
        x *= torch.logspace(-2, 2, shape[-2], device="cuda")[:, None]
    codes = torch.empty(shape, dtype=F8, device="cuda")
    scales = torch.empty(shape[:-2] + (-(-shape[-2] // block), shape[-1] // 128), device="cuda")
    moe.moe_quantize_fp8(x, codes, scales, block_rows=block)
    return codes, scales


def check_product(out, a, sa, b, sb, what="out"):
    ref, bound = og.product(a.view(torch.uint8).cpu().numpy(), sa.cpu().numpy(), b.view(torch.uint8).cpu().numpy(),
                            sb.cpu().numpy())
    within(f64(out), ref, bound + HALF[out.dtype] * (np.abs(ref) + bound), what)


PRODUCTS = [(1, 1, 128), (1, 4096, 7168), (2, 130, 256), (7, 1003, 1408), (12, 256, 512), (13, 384, 640), (16, 100, 2048),
            (25, 576, 1024), (33, 257, 896), (64, 128, 384), (65, 1000, 256), (128, 512, 4096), (129, 640, 1152),
            (300, 1003, 1408), (777, 264, 128), (1500, 2000, 384), (2100, 2304, 512),
            (3000, 1003, 384), (2999, 2308, 128), (1537, 4097, 640)]


@pytest.mark.parametrize("M,N,K", PRODUCTS)
@pytest.mark.parametrize("dtype", [BF, F32])
def test_product(M, N, K, dtype):
    a, sa = codes_of(M, K, block=1, seed=1)
    b, sb = codes_of(N, K, block=128, seed=2)
    out = torch.full((M, N), float("nan"), dtype=dtype, device="cuda")
    status = torch.zeros(1, dtype=I32, device="cuda")
    moe.moe_product_fp8(a, sa, b, sb, out, status=status)
    check_product(out, a, sa, b, sb)
    assert status.item() == 0
    again = torch.empty_like(out)
    moe.moe_product_fp8(a.view(torch.uint8), sa, b.view(torch.uint8), sb, again)
    assert torch.equal(again, out)                                   # equal inputs, equal bits
    # rows apart, and off 16 bytes
    for lead, off in ((16, 0), (3, 1)):
        wide, room = strided(a.view(torch.uint8), K + 16), torch.full((M * (N + lead) + off,), 7.0, dtype=dtype, device="cuda")
        part = room[off:].view(M, N + lead)
        moe.moe_product_fp8(wide, sa, b, sb, part[:, :N])
        assert torch.equal(part[:, :N], out) and (part[:, N:] == 7).all() and (room[:off] == 7).all()


GROUPED = [(3, 2, 8, 256, 128), (64, 8, 256, 128, 256), (40, 4, 16, 200, 384), (200, 4, 8, 384, 512), (300, 2, 4, 1003, 256),
           (700, 2, 4, 640, 1024), (1300, 4, 8, 512, 384), (2500, 2, 3, 768, 256), (600, 8, 2, 257, 640), (4000, 2, 4, 1003, 256),
           (900, 8, 16, 1028, 640), (2100, 8, 3, 640, 128)]


@pytest.mark.parametrize("T,k,E,N,K", GROUPED)
@pytest.mark.parametrize("drop,skew", [(0.0, False), (0.3, True)])
def test_grouped_product(T, k, E, N, K, drop, skew):
    """Groups of all sizes, none among them; rows behind the last one and their NaN stay away."""
    ids = draw_ids(T, k, E, drop, 3, skew)
    offsets = sort_picks(ids, E)["offsets"]
    off = offsets.tolist()
    M = T * k + 5
    a, sa = codes_of(M, K, block=1, seed=1)
    a.view(torch.uint8)[off[-1]:] = 0x7f
    sa[off[-1]:] = float("nan")
    b, sb = codes_of(E, N, K, block=128, seed=2)
    out = torch.full((M, N), 7.0, dtype=BF if T % 200 else F32, device="cuda")
    status = torch.zeros(1, dtype=I32, device="cuda")
    moe.moe_product_fp8(a, sa, b, sb, out, offsets=offsets, status=status)
    assert status.item() == 0
    for e in range(E):
        rows = slice(off[e], off[e + 1])
        if off[e] < off[e + 1]:
            check_product(out[rows], a[rows], sa[rows], b[e], sb[e], "expert %d" % e)
    assert (out[off[-1]:] == 7).all()


@pytest.mark.parametrize("M,N,K", [(5, 384, 256), (200, 256, 640)])
def test_product_gradient_of_the_rows(M, N, K):
    """d(a) of out = a b^T is the product of out's gradient and the transposed codes and scales."""
    dy, sy = codes_of(M, N, block=1, seed=1)
    b, sb = codes_of(N, K, block=128, seed=2)
    da = torch.empty((M, K), device="cuda")
    moe.moe_product_fp8(dy, sy, b.view(torch.uint8).t().contiguous(), sb.t().contiguous(), da)
    w = ofp8.decode_e4m3(b.view(torch.uint8).cpu().numpy()) * np.repeat(np.repeat(f64(sb), 128, 0), 128, 1)
    g = ofp8.decode_e4m3(dy.view(torch.uint8).cpu().numpy()) * np.repeat(f64(sy), 128, 1)
    size = np.abs(g) @ np.abs(w)
    bound = (128 * 2.0 ** -23 + (N // 128 + 5) * EPS32) * size
    within(f64(da), g @ w, bound + EPS32 * size, "da")


def test_product_offsets_of_all_kinds():
    """Rows in front of the first group, empty groups, offsets beyond the rows: as if clamped."""
    M, N, K = 70, 130, 256
    a, sa = codes_of(M, K, block=1, seed=1)
    b, sb = codes_of(5, N, K, block=128, seed=2)
    for off in ([3, 3, 20, 20, 69, 70], [0, 0, 0, 0, 0, 0], [70, 70, 70, 70, 70, 70], [-5, 10, 10, 90, 100, 1 << 30]):
        out = torch.full((M, N), 7.0, device="cuda")
        moe.moe_product_fp8(a, sa, b, sb, out, offsets=torch.tensor(off, dtype=I32, device="cuda"))
        c = [min(max(v, 0), M) for v in off]
        assert (out[:c[0]] == 7).all() and (out[c[-1]:] == 7).all()
        for e in range(5):
            if c[e] < c[e + 1]:
                check_product(out[c[e]:c[e + 1]], a[c[e]:c[e + 1]], sa[c[e]:c[e + 1]], b[e], sb[e])


@pytest.mark.parametrize("M,N", [(70, 130), (900, 2100)])
def test_product_offsets_that_do_not_ascend(M, N):
    """Nothing beyond out is written, and the next call is right."""
    K = 256
    a, sa = codes_of(M, K, block=1, seed=1)
    b, sb = codes_of(9, N, K, block=128, seed=2)
    room = torch.full((3 * M, N), 7.0, device="cuda")
    low, high = -(1 << 31), (1 << 31) - 1
    for off in ([0, M, 0, M, 0, M, 0, M, 0, M], [high, low] * 5, [M, 9, M, 8, M, 7, M, 6, M, 5], [5, 0, 1, 0, 1, 0, 1, 0, 1, 0]):
        moe.moe_product_fp8(a, sa, b, sb, room[M:2 * M], offsets=torch.tensor(off, dtype=I32, device="cuda"))
        assert (room[:M] == 7).all() and (room[2 * M:] == 7).all()
    moe.moe_product_fp8(a, sa, b[:1], sb[:1], room[M:2 * M], offsets=torch.tensor([0, M], dtype=I32, device="cuda"))
    check_product(room[M:2 * M], a, sa, b[0], sb[0])


@pytest.mark.parametrize("M,N,K", [(1, 256, 1024), (200, 300, 512), (1600, 2100, 256)])
def test_product_extremes(M, N, K):
    """Largest codes, scales at both ends of float32, NaN in one row and in one block of weights."""
    a, b = (torch.full(s, 0x7e, dtype=torch.uint8, device="cuda") for s in ((M, K), (N, K)))
    sa, sb = torch.full((M, K // 128), 2.0 ** 60, device="cuda"), torch.full((-(-N // 128), K // 128), 2.0 ** -60, device="cuda")
    out = torch.empty((M, N), device="cuda")
    moe.moe_product_fp8(a, sa, b, sb, out)
    assert torch.equal(out, torch.full_like(out, 448.0 * 448 * K))      # sums of 2^8 * 49 * 2^8: exact
    a[M - 1, 5] = 0x7f
    moe.moe_product_fp8(a, sa, b, sb, out)
    assert out[M - 1].isnan().all() and (out[:M - 1] == 448.0 * 448 * K).all()
    a[M - 1, 5] = 0
    sb[-1, 0] = float("inf")
    moe.moe_product_fp8(a, sa, b, sb, out)
    n = (N - 1) // 128 * 128
    assert out[:, n:].isinf().all() and out[:, :n].isfinite().all()


def test_product_empty():
    b, sb = codes_of(130, 256, block=128, seed=2)
    moe.moe_product_fp8(torch.empty((0, 256), dtype=F8, device="cuda"), torch.empty((0, 2), device="cuda"), b, sb,
                        torch.empty((0, 130), device="cuda"))


# ---- streams, graphs, and the operators together -------------------------------------------------

def chain_inputs(T, H, E, k, I, seed):
    x, ids = rnd(T, H, seed=seed), torch.tensor(draw_ids(T, k, E, 0.1, seed)).cuda()
    w = rnd(T, k, dtype=F32, seed=seed).abs()
    return x, ids, w


class Chain:
    """Experts on sorted rows: quantise, sort, product, SwiGLU, product, and back."""

    def __init__(self, T, H, E, k, I):
        e = lambda *s, dtype=F32: torch.empty(s, dtype=dtype, device="cuda")  # noqa: E731
        P = T * k
        self.E = E
        self.w1, self.s1 = codes_of(E, 2 * I, H, block=128, seed=11)
        self.w2, self.s2 = codes_of(E, H, I, block=128, seed=12)
        self.codes, self.scales = e(T, H, dtype=F8), e(T, H // 128)
        self.offsets, self.position = e(E + 1, dtype=I32), e(T, k, dtype=I32)
        self.work = e(moe.moe_sort_picks_workspace_size(T, k, E), dtype=torch.uint8)
        self.rows, self.rs = e(P, H, dtype=F8), e(P, H // 128)
        self.h, self.act, self.acts, self.y = e(P, 2 * I, dtype=BF), e(P, I, dtype=F8), e(P, I // 128), e(P, H, dtype=BF)
        self.out = e(T, H, dtype=BF)

    def run(self, x, ids, w, stream=None):
        s = dict(stream=stream)
        moe.moe_quantize_fp8(x, self.codes, self.scales, **s)
        moe.moe_sort_picks(ids, self.E, self.offsets, self.position, self.work, **s)
        moe.moe_sort_rows(self.codes, self.position, self.rows, x_scales=self.scales, rows_scales=self.rs, **s)
        moe.moe_product_fp8(self.rows, self.rs, self.w1, self.s1, self.h, offsets=self.offsets, **s)
        moe.moe_swiglu_fp8(self.h, self.act, self.acts, live_rows=self.offsets[-1:], **s)
        moe.moe_product_fp8(self.act, self.acts, self.w2, self.s2, self.y, offsets=self.offsets, **s)
        moe.moe_unsort_rows(self.y, w, self.position, self.out, **s)
        return self.out


@pytest.mark.parametrize("T,H,E,k,I", [(5, 512, 16, 4, 256), (350, 512, 16, 4, 384), (1500, 256, 4, 2, 512)])
def test_chain(T, H, E, k, I):
    """Each step against the oracle from what the step before left; the order is the layer's own."""
    c = Chain(T, H, E, k, I)
    x, ids, w = chain_inputs(T, H, E, k, I, 0)
    out = c.run(x, ids, w)
    codes, scales, _ = ofp8.quantize_rows(f64(x))
    offsets, position, _ = og.order(ids.cpu().numpy(), E)
    np.testing.assert_array_equal(c.position.cpu().numpy(), position)
    n = int(offsets[-1])
    t = np.zeros(n, np.int64)
    for i, p in np.ndenumerate(position):
        if p >= 0:
            t[p] = i[0]
    np.testing.assert_array_equal(c.rows[:n].view(torch.uint8).cpu().numpy(), codes[t])
    np.testing.assert_array_equal(c.rs[:n].cpu().numpy(), scales[t])
    for e in range(E):
        r = slice(int(offsets[e]), int(offsets[e + 1]))
        if r.start < r.stop:
            check_product(c.h[r], c.rows[r], c.rs[r], c.w1[e], c.s1[e], "gate and up")
            check_product(c.y[r], c.act[r], c.acts[r], c.w2[e], c.s2[e], "down")
    ref, bound = og.unsort_rows(np.where(np.arange(len(c.y))[:, None] < n, f64(c.y), 0), f64(w), position)
    within(f64(out), ref, bound + HALF[BF] * (np.abs(ref) + bound), "out")
    layer = moe.MoELayer1GPU(1, T, T, H, E, k, 128, "FLAT", "HT")
    layer.dispatch(x, ids, w)
    assert torch.equal(layer.view("pick_pos", (T, k), torch.int32), c.position)
    assert torch.equal(layer.view("offsets", (E + 1,), torch.int32), c.offsets)


def test_streams_and_graphs():
    """Two chains at once on streams of their own, each captured into a graph and replayed on new
    inputs, give what they give alone."""
    T, H, E, k, I = 200, 512, 8, 2, 256
    cases = [chain_inputs(T, H, E, k, I, s) for s in (1, 2, 3, 4)]
    alone = Chain(T, H, E, k, I)
    want = [alone.run(*c).clone() for c in cases]
    chains, streams = [Chain(T, H, E, k, I) for _ in range(2)], [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(3):
        for i in range(2):
            chains[i].out.fill_(9)
        torch.cuda.synchronize()
        for i in range(2):
            chains[i].run(*cases[i], stream=streams[i])
        torch.cuda.synchronize()
        for i in range(2):
            assert torch.equal(chains[i].out, want[i])
    held, graphs = [[t.clone() for t in cases[i]] for i in range(2)], []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            chains[i].run(*held[i])
        graphs.append(g)
    for turn in (0, 2):
        for i in range(2):
            for to, t in zip(held[i], cases[turn + i]):
                to.copy_(t)
        torch.cuda.synchronize()
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                graphs[i].replay()
        torch.cuda.synchronize()
        for i in range(2):
            assert torch.equal(chains[i].out, want[turn + i])


def test_first_calls_inside_a_capture():
    """A process whose first calls are captured: what is set up once is set up there too."""
    code = """
import sys, torch
sys.path.insert(0, %r)
import combine_topk_ids_gb300 as moe
z = lambda *s, dtype=torch.float32: torch.zeros(s, dtype=dtype, device="cuda")
F8, I32 = torch.float8_e4m3fn, torch.int32
ids, off, pos = torch.randint(0, 1000, (600, 4), device="cuda"), z(1001, dtype=I32), z(600, 4, dtype=I32)
work = z(moe.moe_sort_picks_workspace_size(600, 4, 1000), dtype=torch.uint8)
x, codes, scales = torch.randn(2600, 256, device="cuda"), z(2600, 256, dtype=F8), z(2600, 2)
b, bs, wide, few = torch.ones(2304, 256, device="cuda").to(F8), z(18, 2) + 1, z(2600, 2304), z(3, 2304)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    moe.moe_sort_picks(ids, 1000, off, pos, work)
    moe.moe_quantize_fp8(x, codes, scales)
    moe.moe_product_fp8(codes, scales, b, bs, wide)
    moe.moe_product_fp8(codes[:3], scales[:3], b, bs, few)
for _ in range(2):
    g.replay()
torch.cuda.synchronize()
v = (codes.float() * scales.repeat_interleave(128, 1)).double().sum(1)
assert off[-1] == 2400 and ((wide.double() - v[:, None]).abs() < 1e-3).all() and torch.equal(few, wide[:3])
print("captured")
""" % ROOT
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=200)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]


def test_gradient_reaches_the_router():
    """Combine's gradient in the weights, through the router's, against differences in the logits."""
    T, H, E, k = 4, 64, 8, 2
    router = moe.make_router(E, k, "sigmoid", scale=1.5)
    logits, rows, dout = rnd(T, E, dtype=F32), rnd(T * k, H, dtype=F32), rnd(T, H, dtype=F32, seed=1)
    ids, w, out = torch.empty((T, k), dtype=torch.int64, device="cuda"), torch.empty((T, k), device="cuda"), torch.empty_like(dout)

    def forward():
        moe.moe_route_topk(router, logits, None, ids, w)

    forward()
    position = sort_picks(ids.cpu().numpy(), E)["position"]
    dw, dlogits = torch.empty_like(w), torch.empty_like(logits)
    moe.moe_unsort_rows_backward(dout, rows, w, position, None, dw)
    moe.moe_route_topk_backward(router, logits, ids, dw, dlogits)

    def loss():
        forward()
        moe.moe_unsort_rows(rows, w, position, out)
        return (out.double() * dout.double()).sum().item()

    for t in range(T):
        e, h = int(ids[t, 0]), 2.0 ** -6
        keep, picked = logits[t, e].item(), ids.clone()
        logits[t, e] = keep + h
        up = loss()
        assert torch.equal(ids, picked)
        logits[t, e] = keep - h
        down = loss()
        assert torch.equal(ids, picked)
        logits[t, e] = keep
        # third derivatives of 1.5 * <dout, rows> * share: below 1.5 * |dot| / 6 * h^2; float32 sums over h
        size = 1.5 * (dout[t].abs() * rows.abs().max()).sum().item()
        assert abs((up - down) / (2 * h) - dlogits[t, e].item()) < size * (h * h / 6 + 64 * EPS32 / h)
