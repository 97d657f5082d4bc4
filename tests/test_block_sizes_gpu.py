"""The operators around the expert layer where a block takes several rows or units, one after the
other: the norm's next rows under way while one is computed, the 4-bit experts' ring of stages
filled more than once within a unit.  Against float64 on the GPU, from the formulas."""
import os

import numpy as np
import pytest
import torch

import combine_topk_ids_gb300 as moe
from oracle import fp8 as ofp8

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
EPS32, BF16, E4M3 = 2.0 ** -24, 2.0 ** -8, 2.0 ** -4


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    if not os.path.exists(moe.LIB_PATH):
        moe.build()


def rnd(*shape, dtype=BF, scale=1.0, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def within(got, ref, bound, what):
    bad = ~((got.double() - ref).abs() <= bound)
    assert not bad.any(), "%s: %d of %d outside, first at %s" % (what, bad.sum(), bad.numel(), bad.nonzero()[0].tolist())


# Row groups per block, on 152 SMs: 20011 rows of 256 are 2502 groups of 8, 65536 columns one block an SM.
LONG = [(20011, 256), (1900, 4096), (1300, 7168), (1000, 16384), (700, 65536), (9001, 640)]


@pytest.mark.parametrize("T,H", LONG)
@pytest.mark.parametrize("residual,weight", [(BF, BF), (F32, F32), (None, BF)])
def test_norm_of_many_rows(T, H, residual, weight):
    x = rnd(T, H)
    res = None if residual is None else rnd(T, H, dtype=residual, scale=3, seed=1)
    w = (1 + rnd(H, dtype=F32, scale=0.2, seed=2)).to(weight)
    r = {"sum_out": torch.empty((T, H), dtype=residual or BF, device="cuda"), "rstd": torch.empty(T, device="cuda"),
         "out": torch.empty_like(x), "out_fp8": torch.empty((T, H), dtype=torch.float8_e4m3fn, device="cuda"),
         "scales": torch.empty((T, H // 128), device="cuda")}
    moe.moe_add_rmsnorm(x, res, w, 1e-6, **r)
    h = x.double() if res is None else x.double() + res.double()
    rstd = (h.square().mean(1) + 1e-6).rsqrt()
    # a sum of squares has at most 64 terms in a thread and 37 more additions, half of that after the root
    e = 55 * EPS32
    within(r["rstd"], rstd, (e + 4 * EPS32) * rstd, "rstd")
    within(r["sum_out"], h, ((0 if residual == F32 else BF16) + 2 * EPS32) * h.abs(), "sum")
    y = h * rstd[:, None] * w.double()
    del h
    within(r["out"], y, (BF16 + e + 8 * EPS32) * y.abs(), "out")
    top = y.abs().view(T, -1, 128).amax(2)
    within(r["scales"], top / 448, 2 * (e + 8 * EPS32) * top / 448, "scales")
    sc = r["scales"].double().repeat_interleave(128, 1)
    within(r["out_fp8"].double() * sc, y, (E4M3 + 2 * (e + 8 * EPS32)) * y.abs() + 2.0 ** -10 * 1.001 * sc, "codes")
    del y, sc
    # in place, the same bits
    moe.moe_add_rmsnorm(x, res, w, 1e-6, sum_out=res, out=x)
    assert torch.equal(x.view(torch.int16), r["out"].view(torch.int16))
    assert res is None or torch.equal(res, r["sum_out"])


def test_norm_codes_are_the_dispatch_rules():
    """Rows whose norm is exact in float32 (integers whose squares' sum is H 64^2, weights that are
    powers of two): codes and scales are those of the FP8 dispatch's rule, bit for bit."""
    T, H = 40, 256
    rng = np.random.default_rng(5)
    squares = {}
    for a in range(0, 128):
        for b in range(a, 128):
            squares.setdefault(a * a + b * b, (a, b))
    rows = []
    while len(rows) < T:
        v = rng.integers(-110, 111, H)
        left = H * 64 * 64 - int((v[:-2].astype(np.int64) ** 2).sum())
        if left in squares:
            v[-2:] = squares[left]
            rows.append(v)
        else:   # towards the sum, then again
            while not 0 <= left < 32000:
                i = rng.integers(0, H - 2)
                step = -1 if left < 0 else 1
                if 0 < abs(v[i]) + step < 110:
                    v[i] += step * (1 if v[i] >= 0 else -1)
                left = H * 64 * 64 - int((v[:-2].astype(np.int64) ** 2).sum())
            if left in squares:
                v[-2:] = squares[left]
                rows.append(v)
    v = np.array(rows, dtype=np.float64)
    assert ((v * v).sum(1) == H * 4096).all()
    w = 2.0 ** rng.integers(-3, 4, H)
    q = torch.empty((T, H), dtype=torch.uint8, device="cuda")
    sc, out = torch.empty((T, 2), device="cuda"), torch.empty((T, H), dtype=BF, device="cuda")
    moe.moe_add_rmsnorm(torch.tensor(v).to(BF).cuda(), None, torch.tensor(w, dtype=F32).cuda(), 0.0, out=out,
                        out_fp8=q, scales=sc)
    y = v / 64 * w
    assert (out.cpu().double().numpy() == y).all()
    codes, scales, _ = ofp8.quantize_rows(y.astype(np.float32))
    np.testing.assert_array_equal(q.cpu().numpy(), codes)
    np.testing.assert_array_equal(sc.cpu().numpy(), scales.astype(np.float32))


def unpack(codes, scales):
    v = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).double() - 8
    s = scales.double().repeat_interleave(v.shape[-1] // scales.shape[-1], -1)
    return v * s, s


def w4_reference(x, ids, weights, w1, s1, w2, s2, G):
    """out and the bound of the kernels' arithmetic.  A product's sum is taken in matrix steps of 16
    exact products and a start of -8 times the inputs' sum, each of the 17 truncated to 24 bits
    of the largest (four steps a part: 68 2^-23), and the parts of G or 64 inputs one after the
    other; with code + 8 <= |code - 8| + 16 all of it is relative to (|W| + 16 scale) |x|.  The
    activation is rounded to the 11 bits of f16, or 2^-38 of its row's largest."""
    T, H = x.shape
    I = w2.shape[2] * 2
    out, off = (torch.zeros((T, H), dtype=torch.float64, device="cuda") for _ in range(2))
    c = lambda K: (140 + K / min(G, 64)) * EPS32  # noqa: E731
    for e in sorted(set(ids.flatten().tolist()) - {-1}):
        t, j = (ids == e).nonzero(as_tuple=True)
        up, us = unpack(w1[e], s1[e])
        down, ds = unpack(w2[e], s2[e])
        xt = x[t].double()
        h, dh = xt @ up.T, c(H) * (xt.abs() @ (up.abs() + 16 * us).T)
        g, u, dg, du = h[:, :I], h[:, I:], dh[:, :I], dh[:, I:]
        sg = g * torch.sigmoid(g)
        act = sg * u
        da = 1.1 * dg * (u.abs() + du) + sg.abs() * du + (2.0 ** -11 + 8 * EPS32) * act.abs()
        da += 2.0 ** -38 * act.abs().amax(1, keepdim=True)
        rw = weights[t, j].double()[:, None]
        y, dy = act @ down.T, da @ down.abs().T + c(I) * ((act.abs() + da) @ (down.abs() + 16 * ds).T)
        out.index_add_(0, t, rw * y)
        off.index_add_(0, t, rw.abs() * (dy + (weights.shape[1] + 2) * EPS32 * y.abs()))
    return out, off + BF16 * out.abs() + 2.0 ** -133


def w4_case(T, H, E, k, I, G, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    byte = lambda *s: torch.randint(0, 256, s, generator=g, dtype=torch.uint8, device="cuda")  # noqa: E731
    sc = lambda n, *s: ((torch.rand(s, generator=g, device="cuda") + 0.5) * n).to(BF)  # noqa: E731
    ids = torch.rand((T, E), generator=g, device="cuda").argsort(1)[:, :k].contiguous()
    w = torch.rand((T, k), generator=g, device="cuda") + 0.05
    x = torch.randn((T, H), generator=g, device="cuda").to(BF)
    return (x, ids, w, byte(E, 2 * I, H // 2), sc(0.3 / H ** 0.5, E, 2 * I, H // G), byte(E, H, I // 2),
            sc(0.5 / I ** 0.5, E, H, I // G))


@pytest.mark.parametrize("T,H,E,k,I", [
    (10, 1280, 64, 8, 1152),    # 9 and 10 blocks of 128 inputs; several units to a block in either product
    (4, 2304, 32, 6, 2176),     # 18 and 17
    (40, 1664, 16, 4, 1408),    # several runs of eight picks to an expert
    (2, 4096, 4, 2, 14336),     # 56 stages
    (1, 128, 300, 1, 8192)])
@pytest.mark.parametrize("G", [32, 64, 128])
def test_w4_long_units(T, H, E, k, I, G):
    case = w4_case(T, H, E, k, I, G, seed=T + G)
    layer = moe.MoELayerW4(T, H, E, k, I, G)
    layer.set_weights(*case[3:])
    out = layer.forward(*case[:3]).clone()
    assert layer.status() == 0
    within(out, *w4_reference(*case, G), "out")
    layer.workspace.fill_(255)
    assert torch.equal(layer.forward(*case[:3]), out)      # nothing left over, nothing in another order
    one = [v[:1].contiguous() for v in case[:3]]
    assert torch.equal(layer.forward(*one), out[:1])       # and not by the batch around a token
