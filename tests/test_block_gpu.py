"""The operators around the expert layer on the GPU, through the public entry points, against
the float64 oracle, at the sizes, strides and masks where they can go wrong."""
import numpy as np
import pytest
import torch

import combine_topk_ids_gb300 as moe
from oracle import block as ob

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import os
    if not os.path.exists(moe.LIB_PATH):
        moe.build()


def f64(t):
    return t.detach().cpu().double().numpy()


def rnd(*shape, dtype=BF, scale=1.0, seed=0):
    g = torch.Generator().manual_seed(seed + 1000 * len(shape) + sum(shape))
    return (torch.randn(shape, generator=g) * scale).to(dtype).cuda()


def within(got, ref, bound, what):
    d = np.abs(got - ref)
    bad = ~(d <= bound)
    assert not bad.any(), "%s: %d of %d outside; worst %.3g at %s" % (
        what, bad.sum(), bad.size, d[bad].max(), np.argwhere(bad)[0])


# ---- norm --------------------------------------------------------------------------------------

NORM_SHAPES = [(1, 1), (1, 7168), (3, 128), (5, 7), (7, 2047), (9, 2050), (33, 1000), (17, 4096), (2, 8193),
               (300, 256), (2, 16384), (2, 65536), (2, 65535), (1300, 384)]


def check_norm(x, res, w, eps, r):
    h, rstd, y = ob.add_rmsnorm(f64(x), None if res is None else f64(res), f64(w), eps)
    # sum of squares: at most 64 terms per thread and 37 more additions, half of that after the root
    e = 55 * ob.EPS32
    if r.get("rstd") is not None:
        within(f64(r["rstd"]), rstd, (e + 4 * ob.EPS32) * rstd, "rstd")
    if r.get("sum_out") is not None:
        half = ob.BF16 if r["sum_out"].dtype == BF else 0
        within(f64(r["sum_out"]), h, (half + 2 * ob.EPS32) * np.abs(h) + 1e-38, "sum")
    rel = e + 8 * ob.EPS32
    if r.get("out") is not None:
        within(f64(r["out"]), y, (ob.BF16 + rel) * np.abs(y) + 1e-38, "out")
    if r.get("out_fp8") is not None:
        T, H = x.shape
        top = np.maximum(np.abs(y).reshape(T, H // 128, 128).max(2), 2.0 ** -100)
        within(f64(r["scales"]), top / 448, 2 * rel * top / 448, "scales")
        sc = np.repeat(f64(r["scales"]), 128, 1)
        codes = f64(r["out_fp8"].view(torch.float8_e4m3fn).float())
        # half a code in the normal range, half the smallest step (2^-10) below it
        within(codes * sc, y, (ob.E4M3 + 2 * rel) * np.abs(y) + 2.0 ** -10 * 1.001 * sc, "codes")
        assert np.abs(codes).reshape(T, H // 128, 128).max(2).min() == 448 or np.abs(y).max() == 0


@pytest.mark.parametrize("T,H", NORM_SHAPES)
@pytest.mark.parametrize("residual,weight", [(BF, BF), (None, F32), (F32, F32), (F32, BF)])
def test_norm_forward(T, H, residual, weight):
    x = rnd(T, H)
    res = None if residual is None else rnd(T, H, dtype=residual, scale=3, seed=1)
    w = (1 + rnd(H, dtype=F32, scale=0.2)).to(weight)
    r = {"sum_out": torch.empty((T, H), dtype=residual or BF, device="cuda"), "rstd": torch.empty(T, device="cuda"),
         "out": torch.empty((T, H), dtype=BF, device="cuda")}
    if H % 128 == 0:
        r["out_fp8"] = torch.empty((T, H), dtype=torch.float8_e4m3fn, device="cuda")
        r["scales"] = torch.empty((T, H // 128), device="cuda")
    moe.moe_add_rmsnorm(x, res, w, 1e-6, **r)
    check_norm(x, res, w, 1e-6, r)
    only = {"out": torch.empty_like(r["out"])}
    moe.moe_add_rmsnorm(x, res, w, 1e-6, **only)   # fewer outputs, the same bits
    assert torch.equal(only["out"].view(torch.int16), r["out"].view(torch.int16))
    if H % 128 == 0:
        q = {"out_fp8": torch.empty((T, H), dtype=torch.uint8, device="cuda"), "scales": torch.empty_like(r["scales"])}
        moe.moe_add_rmsnorm(x, res, w, 1e-6, **q)
        assert torch.equal(q["out_fp8"], r["out_fp8"].view(torch.uint8)) and torch.equal(q["scales"], r["scales"])


@pytest.mark.parametrize("T,H,lead,off", [(5, 200, 333, 1), (4, 4096, 5000, 3), (4, 4096, 4104, 8), (3, 507, 512, 5)])
def test_norm_strided_rows_and_in_place(T, H, lead, off):
    """Rows inside wider rows that start anywhere; sum over residual, out over x; the columns
    around the rows keep their values."""
    wide_x, wide_r = rnd(T, lead), rnd(T, lead, seed=1)
    x, res = wide_x[:, off:off + H], wide_r[:, off:off + H]
    w = rnd(H, dtype=BF, seed=2)
    x0, r0, keep = x.clone(), res.clone(), (wide_x.clone(), wide_r.clone())
    ref = {"out": torch.empty((T, H), dtype=BF, device="cuda"), "sum_out": torch.empty((T, H), dtype=BF, device="cuda")}
    moe.moe_add_rmsnorm(x, res, w, 1e-5, **ref)
    check_norm(x0, r0, w, 1e-5, ref)
    moe.moe_add_rmsnorm(x, res, w, 1e-5, sum_out=res, out=x)
    # another start of the rows is another order of a row's sum: the bound, not the bits
    check_norm(x0, r0, w, 1e-5, {"out": x, "sum_out": res})
    for wide, k in ((wide_x, keep[0]), (wide_r, keep[1])):
        assert torch.equal(wide[:, :off], k[:, :off]) and torch.equal(wide[:, off + H:], k[:, off + H:])


def test_norm_special_rows():
    H = 256
    x = rnd(6, H)
    x[1] = 0
    x[2, 5] = float("nan")
    x[3, 7] = float("inf")
    x[4] *= 1e-30
    out, q = torch.empty_like(x), torch.empty((6, H), dtype=torch.float8_e4m3fn, device="cuda")
    sc = torch.empty((6, 2), device="cuda")
    w = torch.ones(H, device="cuda")
    moe.moe_add_rmsnorm(x, None, w, 1e-6, out=out, out_fp8=q, scales=sc)
    o = out.float()
    assert (o[1] == 0).all() and (q[1].float() == 0).all() and (sc[1] == 2.0 ** -100 / 448).all()
    assert o[2].isnan().all() and o[3, 7].isnan() and (o[3, :7] == 0).all()
    for t in (0, 4, 5):
        check_norm(x[t:t + 1], None, w, 1e-6, {"out": out[t:t + 1], "out_fp8": q[t:t + 1], "scales": sc[t:t + 1]})
    empty = torch.empty((0, H), dtype=BF, device="cuda")
    moe.moe_add_rmsnorm(empty, empty, w, 1e-6, sum_out=empty, out=empty)


@pytest.mark.parametrize("T,H", [(1, 1), (1, 7168), (5, 7), (7, 2047), (33, 1000), (700, 256), (650, 4096),
                                 (3, 8200), (2, 65536)])
@pytest.mark.parametrize("stream,weight,dsum", [(BF, BF, True), (F32, F32, True), (BF, F32, False)])
def test_norm_backward(T, H, stream, weight, dsum):
    h = rnd(T, H, dtype=stream, scale=2)
    w = (1 + rnd(H, dtype=F32, scale=0.2)).to(weight)
    rstd = torch.rsqrt(h.double().square().mean(1) + 1e-6).float()
    dout = rnd(T, H, seed=3)
    ds = rnd(T, H, dtype=stream, seed=4) if dsum else None
    dx = torch.empty((T, H), dtype=stream, device="cuda")
    dw = torch.empty(H, device="cuda")
    ws = torch.empty(moe.moe_add_rmsnorm_workspace_size(T, H), dtype=torch.uint8, device="cuda")
    moe.moe_add_rmsnorm_backward(dout, h, w, rstd, dx, dw, ws, dsum=ds)
    rx, rw, bx, bw = ob.add_rmsnorm_backward(f64(dout), f64(h), f64(w), f64(rstd), None if ds is None else f64(ds))
    within(f64(dx), rx, bx + (ob.BF16 if stream == BF else 0) * np.abs(rx) + 1e-38, "dx")
    within(f64(dw), rw, bw + 1e-38, "dweight")
    first = dw.clone()
    ws.fill_(255)
    if ds is not None:   # in place over dsum
        moe.moe_add_rmsnorm_backward(dout, h, w, rstd, ds, dw, ws, dsum=ds)
        assert torch.equal(ds, dx)
    else:
        moe.moe_add_rmsnorm_backward(dout, h, w, rstd, dx, dw, ws)
    assert torch.equal(dw, first)   # the same order of sums every time


@pytest.mark.parametrize("T,H,lead,off", [
    (700, 257, (257, 257, 257), (0, 0, 0)),       # more rows than blocks, each off a boundary in its own way
    (5000, 133, (133, 133, 133), (0, 0, 0)),      # the same with several rows in a block
    (650, 4097, (4097, 4097, 4097), (0, 0, 0)),
    (330, 8201, (8203, 8203, 8203), (1, 1, 1)),
    (950, 8201, (8201, 8201, 8201), (0, 0, 0)),   # four rows to some blocks
    (950, 8208, (8208, 8216, 8208), (0, 0, 0)),   # on the boundaries
    (611, 512, (513, 640, 640), (1, 0, 0)),       # dout alone is off the boundaries
    (611, 512, (640, 513, 515), (0, 1, 3)),       # all but dout
    (611, 512, (517, 521, 640), (5, 2, 8)),       # each otherwise
    (9, 5, (5, 9, 6), (0, 4, 1))])
@pytest.mark.parametrize("stream", [BF, F32])
def test_norm_backward_strided_rows(T, H, lead, off, stream):
    """Rows inside wider rows that start anywhere (dout's, h's, and those of dsum, which dx takes
    the place of); the columns around them keep their values."""
    wide = [rnd(T, lead[0], seed=3), rnd(T, lead[1], dtype=stream, scale=2, seed=1),
            rnd(T, lead[2], dtype=stream, seed=4)]
    dout, h, ds = (m[:, o:o + H] for m, o in zip(wide, off))
    keep = [m.clone() for m in wide]
    w = 1 + rnd(H, dtype=F32, scale=0.2, seed=2)
    rstd = torch.rsqrt(h.double().square().mean(1) + 1e-6).float()
    dw = torch.empty(H, device="cuda")
    ws = torch.full((moe.moe_add_rmsnorm_workspace_size(T, H),), 255, dtype=torch.uint8, device="cuda")
    rx, rw, bx, bw = ob.add_rmsnorm_backward(f64(dout), f64(h), f64(w), f64(rstd), f64(ds))
    moe.moe_add_rmsnorm_backward(dout, h, w, rstd, ds, dw, ws, dsum=ds)
    within(f64(ds), rx, bx + (ob.BF16 if stream == BF else 0) * np.abs(rx) + 1e-38, "dx")
    within(f64(dw), rw, bw + 1e-38, "dweight")
    assert torch.equal(wide[0], keep[0]) and torch.equal(wide[1], keep[1])
    assert torch.equal(wide[2][:, :off[2]], keep[2][:, :off[2]])
    assert torch.equal(wide[2][:, off[2] + H:], keep[2][:, off[2] + H:])


def test_norm_backward_against_differences():
    """The GPU's gradient against central differences of the float64 forward."""
    T, H, eps, step = 3, 40, 1e-6, 1e-6
    x, res = f64(rnd(T, H)), f64(rnd(T, H, seed=1))
    w, c = f64(rnd(H, dtype=F32, seed=2)), f64(rnd(T, H, seed=3))
    h, rstd, _ = ob.add_rmsnorm(x, res, w, eps)
    cu = lambda a, dt: torch.tensor(a).to(dt).cuda()  # noqa: E731
    dx, dw = torch.empty((T, H), device="cuda"), torch.empty(H, device="cuda")
    ws = torch.empty(moe.moe_add_rmsnorm_workspace_size(T, H), dtype=torch.uint8, device="cuda")
    moe.moe_add_rmsnorm_backward(cu(c, BF), cu(h, F32), cu(w, F32), cu(rstd, F32), dx, dw, ws)

    def loss(x, w):
        return (ob.add_rmsnorm(x, res, w, eps)[2] * c).sum()

    for i in (0, 13, 39):
        d = np.zeros((T, H))
        d[1, i] = step
        assert abs((loss(x + d, w) - loss(x - d, w)) / (2 * step) - dx[1, i].item()) < 2e-5
        e = np.zeros(H)
        e[i] = step
        assert abs((loss(x, w + e) - loss(x, w - e)) / (2 * step) - dw[i].item()) < 2e-5


def test_norm_empty_batch_backward():
    H = 256
    e = torch.empty((0, H), dtype=BF, device="cuda")
    dw = torch.full((H,), 3.0, device="cuda")
    ws = torch.full((moe.moe_add_rmsnorm_workspace_size(0, H),), 255, dtype=torch.uint8, device="cuda")
    moe.moe_add_rmsnorm_backward(e, e, torch.ones(H, device="cuda"), torch.empty(0, device="cuda"), e, dw, ws)
    assert (dw == 0).all()


# ---- router --------------------------------------------------------------------------------------

ROUTES = [  # T, E, k, rule
    (1, 1, 1, {}), (3, 4, 2, {}), (5, 8, 8, {"renorm": False}), (7, 31, 5, {"kind": "sigmoid"}),
    (33, 60, 4, {"kind": "sigmoid", "bias": True, "scale": 2.5}),
    (65, 72, 6, {"bias": True, "groups": 8, "top_groups": 3}),
    (64, 256, 8, {"kind": "sigmoid", "bias": True, "groups": 8, "top_groups": 4, "pair": True, "scale": 2.5}),
    (64, 256, 8, {"groups": 8, "top_groups": 4}), (19, 160, 6, {"groups": 8, "top_groups": 3, "renorm": False}),
    (40, 128, 4, {}), (9, 384, 8, {"kind": "sigmoid", "bias": True}), (9, 513, 16, {"bias": True}),
    (5, 1000, 32, {"kind": "sigmoid", "groups": 4, "top_groups": 2, "pair": True}),
    (4, 2048, 32, {"groups": 32, "top_groups": 5, "pair": True, "bias": True}), (6, 2047, 8, {}),
    (12, 32, 3, {"groups": 32, "top_groups": 9, "pair": True}),
]


def route_case(T, E, rule, dtype, masked):
    rule = dict(rule)
    bias = torch.round(rnd(E, dtype=F32, seed=5) * 64) / 640 if rule.pop("bias", False) else None
    logits = rnd(T, E, dtype=F32, scale=1.5, seed=6)
    logits = (torch.round(logits * 16) / 16).to(dtype)      # equal values among them
    if masked:
        inf = float("inf")
        for t in range(T):
            logits[t, t % E] = (-inf, float("nan"), inf, torch.finfo(dtype).min, -0.0)[t % 5]
        logits[T // 2] = -inf                               # a token with no expert
        logits[T // 3, 1:] = -inf                           # and one with a single one
    return logits, bias, rule


@pytest.mark.parametrize("T,E,k,rule", ROUTES)
@pytest.mark.parametrize("dtype,ids_dtype,masked", [(F32, torch.int64, False), (BF, torch.int32, True),
                                                    (F32, torch.int32, True)])
def test_route_forward_and_backward(T, E, k, rule, dtype, ids_dtype, masked):
    logits, bias, rule = route_case(T, E, rule, dtype, masked)
    ref_ids, ref_w, gap = ob.route(f64(logits), None if bias is None else f64(bias), k, **rule)
    kind, renorm, scale = rule.get("kind", "softmax"), rule.get("renorm", True), rule.get("scale", 1.0)
    r = moe.make_router(E, k, kind, rule.get("groups", 1), rule.get("top_groups", 1),
                        "top2" if rule.get("pair") else "max", renorm, scale)
    ids = torch.full((T, k), 77, dtype=ids_dtype, device="cuda")
    w = torch.full((T, k), 77.0, device="cuda")
    moe.moe_route_topk(r, logits, bias, ids, w)
    clear = gap > 2e-6      # float32 scores tell these tokens' keys apart
    assert clear.sum() >= 0.9 * T
    np.testing.assert_array_equal(ids.cpu().numpy()[clear], ref_ids[clear])
    within(f64(w)[clear], ref_w[clear], 60 * ob.EPS32 * ref_w[clear] + 1e-37, "weights")
    dw = rnd(T, k, dtype=F32, seed=7)
    dl = torch.full((T, E), 77.0, dtype=dtype, device="cuda")
    moe.moe_route_topk_backward(r, logits, ids, dw, dl)
    ref, bound = ob.route_backward(f64(logits), ids.cpu().numpy(), f64(dw), kind, renorm, scale)
    within(f64(dl), ref, bound + (ob.BF16 if dtype == BF else 0) * np.abs(ref) + 1e-37, "dlogits")


def test_route_lowest_finite_mask_is_a_logit():
    """Experts masked by the type's lowest value stay pickable behind the others; where all
    are, they are equal."""
    E, k = 64, 4
    logits = torch.full((2, E), torch.finfo(F32).min, device="cuda")
    logits[0, 9], logits[0, 3] = 1.0, 2.0
    ids, w = torch.empty((2, k), dtype=torch.int64, device="cuda"), torch.empty((2, k), device="cuda")
    moe.moe_route_topk(moe.make_router(E, k), logits, None, ids, w)
    assert ids.tolist() == [[3, 9, 0, 1], [0, 1, 2, 3]]
    assert w[0, 2:].tolist() == [0, 0] and w[1].tolist() == [0.25] * 4


def test_route_strided_logits_and_empty():
    wide = rnd(9, 300, dtype=F32)
    r = moe.make_router(100, 5)
    got, want = [(torch.empty((9, 5), dtype=torch.int32, device="cuda"), torch.empty((9, 5), device="cuda"))
                 for _ in range(2)]
    moe.moe_route_topk(r, wide[:, 7:107], None, *got)
    moe.moe_route_topk(r, wide[:, 7:107].contiguous(), None, *want)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert r.logits_stride == 0
    a, b = torch.empty((9, 100), device="cuda"), torch.empty((9, 100), device="cuda")
    moe.moe_route_topk_backward(r, wide[:, 7:107], got[0], got[1], a)
    moe.moe_route_topk_backward(r, wide[:, 7:107].contiguous(), got[0], got[1], b)
    assert torch.equal(a, b)
    moe.moe_route_topk(r, wide[:0, :100], None, got[0][:0], got[1][:0])
    moe.moe_route_topk_backward(r, wide[:0, :100], got[0][:0], got[1][:0], a[:0])


@pytest.mark.parametrize("kind,renorm", [("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)])
def test_route_backward_against_differences(kind, renorm):
    T, E, k, step = 2, 10, 3, 1e-6
    logits = rnd(T, E, dtype=F32, seed=8)
    c = rnd(T, k, dtype=F32, seed=9)
    r = moe.make_router(E, k, kind, renormalize=renorm, scale=1.5)
    ids, w = torch.empty((T, k), dtype=torch.int64, device="cuda"), torch.empty((T, k), device="cuda")
    moe.moe_route_topk(r, logits, None, ids, w)
    dl = torch.empty((T, E), device="cuda")
    moe.moe_route_topk_backward(r, logits, ids, c, dl)
    i = ids.cpu().numpy()
    for t in range(T):
        for e in range(E):
            d = np.zeros((T, E))
            d[t, e] = step
            up, down = (ob.route_weights(f64(logits) + s * d, i, kind, renorm, 1.5) for s in (1, -1))
            assert abs(((up - down) * f64(c)).sum() / (2 * step) - dl[t, e].item()) < 1e-6


# ---- 4-bit experts ---------------------------------------------------------------------------------


def w4_case(T, H, E, k, I, G, seed=0):
    g = torch.Generator().manual_seed(seed)
    byte = lambda *s: torch.randint(0, 256, s, generator=g, dtype=torch.uint8).cuda()  # noqa: E731
    sc = lambda n, *s: ((torch.rand(s, generator=g) + 0.5) * n).to(BF).cuda()  # noqa: E731
    ids = torch.rand((T, E), generator=g).argsort(1)[:, :k].contiguous()
    w = torch.rand((T, k), generator=g) + 0.05
    x = torch.randn((T, H), generator=g).to(BF)
    return (x.cuda(), ids.cuda(), w.cuda(), byte(E, 2 * I, H // 2), sc(0.3 / H ** 0.5, E, 2 * I, H // G),
            byte(E, H, I // 2), sc(0.5 / I ** 0.5, E, H, I // G))


def w4_layer(T, H, E, k, I, G, case):
    layer = moe.MoELayerW4(T, H, E, k, I, G)
    layer.set_weights(*case[3:])
    return layer


def check_w4(out, x, ids, w, rest):
    ref, bound = ob.forward_w4(f64(x), ids.cpu().numpy(), f64(w), rest[0].cpu().numpy(), f64(rest[1]),
                               rest[2].cpu().numpy(), f64(rest[3]))
    within(f64(out), ref, bound, "out")


W4_SHAPES = [(1, 128, 1, 1, 128, 128), (1, 256, 8, 2, 128, 64), (3, 256, 8, 2, 512, 32), (2, 640, 5, 3, 384, 128),
             (5, 1152, 16, 4, 256, 32), (9, 128, 1, 1, 256, 64), (17, 256, 2, 1, 128, 32), (40, 256, 1, 1, 256, 128),
             (33, 384, 4, 4, 128, 64), (64, 256, 60, 8, 128, 128), (70, 128, 2, 2, 384, 32), (1, 2048, 128, 8, 1024, 128),
             (4, 1280, 2048, 32, 128, 32)]


@pytest.mark.parametrize("T,H,E,k,I,G", W4_SHAPES)
def test_w4_forward(T, H, E, k, I, G):
    case = w4_case(T, H, E, k, I, G)
    layer = w4_layer(T, H, E, k, I, G, case)
    x, ids, w = case[:3]
    out = layer.forward(x, ids, w).clone()
    assert layer.status() == 0
    check_w4(out, x, ids, w, case[3:])
    layer.workspace.fill_(255)      # nothing is kept in the workspace
    assert torch.equal(layer.forward(x, ids.int(), w), out)
    if T > 2:                       # a smaller batch in the same layer: the same rows
        assert torch.equal(layer.forward(x[:T - 2], ids[:T - 2].contiguous(), w[:T - 2]), out[:T - 2])


def test_w4_masks_and_bad_ids():
    T, H, E, k, I, G = 12, 256, 6, 3, 256, 64
    case = w4_case(T, H, E, k, I, G)
    layer = w4_layer(T, H, E, k, I, G, case)
    x, ids, w = case[:3]
    ids[0] = -1                             # a token with no pick
    ids[1, 1] = -1
    ids[2] = ids[2, 0]                      # one expert three times
    ids[3:9] = torch.tensor([2, 4, 5])      # many rows on three experts
    w[1, 1] = float("nan")                  # a masked pick's weight is not read into the sum
    layer.forward(x, ids, w)
    assert layer.status() == 0
    clean = torch.where(ids < 0, torch.zeros_like(w), w)
    check_w4(layer.out, x, ids, clean, case[3:])
    assert (layer.out[0] == 0).all()
    ids[4, 0], ids[5, 2] = E, -2            # dropped, and reported
    layer.forward(x, ids, w)
    assert layer.status() == moe.STATUS_BAD_EXPERT_ID
    ids[4, 0], ids[5, 2] = -1, -1
    check_w4(layer.out, x, ids, clean, case[3:])
    layer.forward(x, torch.full_like(ids, -1), w)
    assert layer.status() == 0 and (layer.out == 0).all()
    assert layer.forward(x[:0], ids[:0], w[:0]).shape == (0, H) and layer.status() == 0


def test_w4_another_stream_and_graph():
    T, H, E, k, I, G = 6, 512, 8, 2, 256, 32
    case = w4_case(T, H, E, k, I, G)
    layer = w4_layer(T, H, E, k, I, G, case)
    x, ids, w = case[:3]
    want = layer.forward(x, ids, w).clone()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    layer.out.zero_()
    s.wait_stream(torch.cuda.current_stream())
    layer.forward(x, ids, w, stream=s)
    s.synchronize()
    assert torch.equal(layer.out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer.forward(x, ids, w)
    x.copy_(rnd(T, H, seed=11))
    ids.copy_(ids.flip(0))
    graph.replay()
    torch.cuda.synchronize()
    check_w4(layer.out, x, ids, w, case[3:])


@pytest.mark.parametrize("G", [32, 64, 128])
def test_w4_quantize(G):
    w = rnd(37, 384, scale=0.05)
    w[3, :128] = 0
    w[5, 7] = 3.0
    codes = torch.empty((37, 192), dtype=torch.uint8, device="cuda")
    scales = torch.empty((37, 384 // G), dtype=BF, device="cuda")
    moe.moe_quantize_w4(w, G, codes, scales)
    v, sc, c = f64(w).reshape(37, -1, G), f64(scales)[:, :, None], codes.cpu().numpy()
    top = np.abs(v).max(2)
    within(sc[:, :, 0], top / 7, (ob.BF16 + 2 * ob.EPS32) * top / 7, "scales")
    back = ob.unpack_w4(c, f64(scales)).reshape(v.shape)
    # half a step, and where bf16 rounded the scale down, what amax / scale exceeds 7.5 by: nothing
    within(back, v, (0.5 + 1e-5) * sc * np.ones_like(v), "weights")
    assert (c[3, :64] == 0x88).all() and (f64(scales)[3, :128 // G] == 0).all()


def test_w4_against_the_bf16_layer():
    """MoELayerW4 on quantised weights against MoELayer1GPU on the weights they stand for
    (scales that are powers of two, so that those are bf16 values)."""
    T, H, E, k, I, G = 20, 256, 8, 2, 256, 64
    x, ids, w, w1, s1, w2, s2 = w4_case(T, H, E, k, I, G)
    s1, s2 = torch.full_like(s1, 2.0 ** -6), torch.full_like(s2, 2.0 ** -5)
    full = [torch.tensor(ob.unpack_w4(c.cpu().numpy(), f64(s))).to(BF).cuda() for c, s in ((w1, s1), (w2, s2))]
    a = moe.MoELayer1GPU(2, 16, T, H, E, k, I, "EM", "LL")
    a.set_weights(*full)
    b = moe.MoELayerW4(T, H, E, k, I, G)
    b.set_weights(w1, s1, w2, s2)
    ref, bound = ob.forward_w4(f64(x), ids.cpu().numpy(), f64(w), w1.cpu().numpy(), f64(s1), w2.cpu().numpy(), f64(s2))
    within(f64(a.forward(x, ids, w)), ref, bound, "bf16 layer")
    within(f64(b.forward(x, ids, w)), ref, bound, "4-bit layer")


def test_w4_rows_of_all_sizes():
    """Outliers, tiny and empty rows; a row that is not finite spoils its own token alone."""
    T, H, E, k, I, G = 9, 512, 4, 2, 256, 32
    case = w4_case(T, H, E, k, I, G, seed=3)
    layer = w4_layer(T, H, E, k, I, G, case)
    x, ids, w = case[:3]
    x[0] = 0
    x[1, 7] = 3e4
    x[2] *= 1e-12
    x[3, ::2] *= 1e-6
    x[4] *= 1e5
    layer.forward(x, ids, w)
    check_w4(layer.out, x, ids, w, case[3:])
    assert (layer.out[0] == 0).all()
    want = layer.out.clone()
    x[5, 3], x[6, 100] = float("nan"), float("inf")
    out = layer.forward(x, ids, w)
    assert out[5].isnan().all() and out[6].isnan().all() and layer.status() == 0
    keep = [t for t in range(T) if t not in (5, 6)]
    assert torch.equal(out[keep], want[keep])


def test_w4_many_picks():
    """More picks than the blocks count places for themselves, and many rows for each expert."""
    T, H, E, k, I, G = 310, 256, 6, 4, 128, 64
    case = w4_case(T, H, E, k, I, G, seed=5)
    layer = w4_layer(T, H, E, k, I, G, case)
    x, ids, w = case[:3]
    ids[::7, 1] = -1
    out = layer.forward(x, ids, w).clone()
    assert layer.status() == 0
    check_w4(out, x, ids, torch.where(ids < 0, torch.zeros_like(w), w), case[3:])
    assert torch.equal(layer.forward(x[:200], ids[:200].contiguous(), w[:200]), out[:200])
