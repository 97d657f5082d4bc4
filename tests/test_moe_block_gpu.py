"""The operators together, as examples/moe_block.py runs them, and the FP8 dispatch of rows
that are quantised already."""
import os
import sys

import numpy as np
import pytest
import torch

import combine_topk_ids_gb300 as moe
import gen
from gen.device import make_case
from oracle import block as ob
from oracle import fp8 as ofp8

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import moe_block  # noqa: E402

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    if not os.path.exists(moe.LIB_PATH):
        moe.build()


def f64(t):
    return t.detach().cpu().double().numpy()


@pytest.mark.parametrize("name", ["small_em", "small_rm", "small_flat"])
def test_dispatch_of_quantised_rows(name):
    """Rows quantised before the dispatch by the dispatch's own rule: the same layer, bit for bit."""
    cfg = gen.SMALL[name].with_(quant="fp8")
    case = make_case(cfg, "cuda:0")
    layer = moe.MoELayer1GPU(cfg.W, cfg.Tr, cfg.tokens, cfg.H, cfg.E, cfg.k, cfg.I, cfg.layout, cfg.algo, quant="fp8")
    layer.set_weights(case.w1, case.w2)
    want = layer.forward(case.x, case.ids, case.w).clone()
    codes, scales, _ = ofp8.quantize_rows(f64(case.x).astype(np.float32))
    codes, scales = torch.tensor(codes).cuda(), torch.tensor(scales.astype(np.float32)).cuda()
    layer.workspace.zero_()
    layer.expert_out.fill_(7)
    layer.dispatch_fp8(codes, scales, case.ids, case.w)
    layer.expert_ffn()
    assert torch.equal(layer.combine(case.w), want) and layer.status() == 0
    layer.dispatch_fp8(codes.view(torch.float8_e4m3fn), scales, case.ids, case.w, torch.ones(cfg.W, dtype=torch.int32, device="cuda"))
    layer.expert_ffn()
    assert torch.equal(layer.combine(case.w), want)


def parts(T, H, E, k, seed=3):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    norm, gate = (r(H) * 0.1 + 1).to(BF).cuda(), (r(E, H) * H ** -0.5).to(BF).cuda()
    bias = (r(E) * 0.05).cuda()
    x, res = r(T, H).to(BF).cuda(), (2 * r(T, H)).to(BF).cuda()
    return norm, gate, bias, x, res


def test_decode_block():
    """h, y, ids, weights and the output, each against the oracle from what the step before left."""
    T, H, E, k, I = 5, 512, 16, 4, 256
    norm, gate, bias, x, res = parts(T, H, E, k)
    router = moe.make_router(E, k, "sigmoid", 4, 2, "top2", True, 2.5)
    experts = moe.MoELayerW4(T, H, E, k, I, 64)
    w1, w2 = (torch.randn(s, device="cuda").mul_(0.05).to(BF) for s in ((E, 2 * I, H), (E, H, I)))
    experts.quantize_weights(w1, w2)
    codes = []
    for w in (w1, w2):
        c = torch.empty(w.shape[:2] + (w.shape[2] // 2,), dtype=torch.uint8, device="cuda")
        s = torch.empty(w.shape[:2] + (w.shape[2] // 64,), dtype=BF, device="cuda")
        moe.moe_quantize_w4(w, 64, c, s)
        codes += [c.cpu().numpy(), f64(s)]
    x0, r0 = f64(x), f64(res)
    block = moe_block.MoEBlock(T, norm, gate, bias, router)
    out = block.decode(x, res, experts)
    h, _, y = ob.add_rmsnorm(x0, r0, f64(norm), moe_block.EPS)
    assert (np.abs(f64(res) - h) <= 2 * ob.BF16 * np.abs(h) + 1e-30).all()
    assert (np.abs(f64(block.y) - y) <= 2 * ob.BF16 * np.abs(y)).all()
    ids, w, gap = ob.route(f64(block.logits), f64(bias), k, "sigmoid", 4, 2, True, True, 2.5)
    assert (gap > 2e-6).all()
    np.testing.assert_array_equal(block.ids.cpu().numpy(), ids)
    np.testing.assert_allclose(f64(block.weights), w, rtol=1e-5)
    ref, bound = ob.forward_w4(f64(block.y), ids, f64(block.weights), *codes)
    assert (np.abs(f64(out) - ref) <= bound).all() and experts.status() == 0


def test_prefill_block_and_its_gradients():
    """The FP8 prefill: its codes against the float64 norm, its output the layer's own from
    these; and the gradients against autograd in float64."""
    cfg = gen.SMALL["small_flat"].with_(quant="fp8")
    T, H, E, k = cfg.tokens, cfg.H, cfg.E, cfg.k
    norm, gate, bias, x, res = parts(T, H, E, k)
    router = moe.make_router(E, k, "softmax", renormalize=True)
    case = make_case(cfg, "cuda:0")
    layer = moe.MoELayer1GPU(cfg.W, cfg.Tr, T, H, E, k, cfg.I, cfg.layout, cfg.algo, quant="fp8")
    layer.set_weights(case.w1, case.w2)
    block = moe_block.MoEBlock(T, norm, gate, bias, router)
    h0 = res.clone()
    out = block.prefill(x, res, layer).clone()
    assert layer.status() == 0 and (block.ids >= 0).all()
    _, _, y = ob.add_rmsnorm(f64(x), f64(h0), f64(norm), moe_block.EPS)
    sc = np.repeat(f64(block.scales), 128, 1)
    rows = f64(block.codes.float()) * sc
    assert (np.abs(rows - y) <= (ob.E4M3 + 1e-5) * np.abs(y) + 2.0 ** -10 * 1.001 * sc).all()
    layer.out.zero_()
    layer.dispatch_fp8(block.codes, block.scales, block.ids, block.weights)
    layer.expert_ffn()
    assert torch.equal(layer.combine(block.weights), out) and out.float().norm() > 0

    dw = torch.randn((T, k), device="cuda")
    dy = torch.randn((T, H), device="cuda").to(BF)
    dr = torch.randn((T, H), device="cuda").to(BF)
    dx, dnorm, dgate = block.backward(res, dw, dy, dr)
    hh = res.double().requires_grad_()          # the saved stream
    n64, g64 = norm.double().requires_grad_(), gate.double().requires_grad_()
    y = hh * torch.rsqrt(hh.square().mean(1, keepdim=True) + moe_block.EPS) * n64
    w = torch.softmax((y @ g64.T).gather(1, block.ids), 1)
    ((w * dw).sum() + (y * dy).sum() + (hh * dr).sum()).backward()
    # bf16 logits gradients, products and results: a few bf16 roundings of the largest terms
    for got, want in ((dx, hh.grad), (dnorm, n64.grad), (dgate, g64.grad)):
        d = (got.double() - want).norm() / want.norm()
        assert d < 4 * 2.0 ** -8, d
    assert not torch.equal(h0, res)
