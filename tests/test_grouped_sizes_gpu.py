"""The operators on expert-grouped rows at sizes beyond 31 bits of elements, and the example that
runs them together."""
import os
import sys

import numpy as np
import pytest
import torch

import combine_topk_ids_gb300 as moe
import gen
from oracle import fp8 as ofp8
from oracle import grouped as og
from oracle.block import BF16, EPS32

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import grouped_experts  # noqa: E402

pytestmark = pytest.mark.gpu
BF, F32, I32, F8 = torch.bfloat16, torch.float32, torch.int32, torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    if not os.path.exists(moe.LIB_PATH):
        moe.build()


def f64(t):
    return t.detach().cpu().double().numpy()


def test_rows_beyond_31_bits():
    """2.4 G elements of sorted rows: what lies first and last in them."""
    T, k, H = 37500, 8, 8064
    ids = torch.arange(k, device="cuda").repeat(T, 1).roll(3, 1).contiguous()   # pick j has expert (j - 3) % 8
    position = torch.empty((T, k), dtype=I32, device="cuda")
    offsets, source = torch.empty(k + 1, dtype=I32, device="cuda"), torch.empty(T * k, dtype=I32, device="cuda")
    work = torch.empty(moe.moe_sort_picks_workspace_size(T, k, k), dtype=torch.uint8, device="cuda")
    moe.moe_sort_picks(ids, k, offsets, position, work, source=source)
    assert offsets.tolist() == [T * e for e in range(k + 1)]
    want = (torch.arange(T, device="cuda")[:, None] + T * ((torch.arange(k, device="cuda") - 3) % k)[None]).int()
    assert torch.equal(position, want)
    x = torch.arange(T, device="cuda").remainder(251)[:, None].to(BF).expand(T, H).contiguous()
    rows = torch.empty((T * k, H), dtype=BF, device="cuda")
    moe.moe_sort_rows(x, position, rows)
    for e in range(k):
        assert torch.equal(rows[T * e:T * (e + 1)], x)
    w = torch.full((T, k), 0.125, device="cuda")
    out, dw = torch.empty_like(x), torch.empty_like(w)
    moe.moe_unsort_rows(rows, w, position, out)
    assert torch.equal(out, x)                      # eight equal rows at an eighth: exact
    rows.fill_(7)
    moe.moe_unsort_rows_backward(x, rows, w, position, None, dw)
    assert torch.equal(dw, (x[:, :1].float() * 7 * H).expand(T, k))   # integers below 2^24: exact
    moe.moe_unsort_rows_backward(x, None, w, position, rows, None)
    for e in range(k):
        assert torch.equal(rows[T * e:T * (e + 1)], (x.float() / 8).to(BF))


@pytest.mark.parametrize("grouped", [False, True])
def test_product_beyond_31_bits(grouped):
    """2.2 G elements of out; rows from all over it against the oracle."""
    M, N, K = 560000, 3968, 128
    g = torch.Generator(device="cuda").manual_seed(0)
    a = torch.randn((M, K), generator=g, device="cuda", dtype=BF).to(F8)
    sa = torch.rand((M, 1), generator=g, device="cuda") + 0.5
    G = 3 if grouped else 1
    b = torch.randn((G, N, K), generator=g, device="cuda", dtype=BF).to(F8)
    sb = torch.rand((G, N // 128, 1), generator=g, device="cuda") + 0.5
    out = torch.empty((M, N), dtype=BF, device="cuda")
    off = [0, 100001, 100001, M] if grouped else [0, M]
    moe.moe_product_fp8(a, sa, b if grouped else b[0], sb if grouped else sb[0], out,
                        offsets=torch.tensor(off, dtype=I32, device="cuda") if grouped else None)
    for e in range(G):
        for first in {off[e], (off[e] + off[e + 1]) // 2, max(off[e], off[e + 1] - 60)}:
            r = slice(first, min(first + 60, off[e + 1]))
            if r.start >= r.stop:
                continue
            ref, bound = og.product(a[r].view(torch.uint8).cpu().numpy(), sa[r].cpu().numpy(),
                                    b[e].view(torch.uint8).cpu().numpy(), sb[e].cpu().numpy())
            assert (np.abs(f64(out[r]) - ref) <= bound + BF16 * (np.abs(ref) + bound)).all(), (e, first)


def test_weights_of_many_groups():
    """Weight rows beyond 2^31 bytes, most groups empty."""
    E, N, K = 600, 4096, 1024
    b = torch.zeros((E, N, K), dtype=torch.uint8, device="cuda")
    sb = torch.ones((E, N // 128, K // 128), device="cuda")
    last = torch.randn((N, K), device="cuda", dtype=BF).to(F8)
    b[E - 1] = last.view(torch.uint8)
    a = torch.randn((7, K), device="cuda", dtype=BF).to(F8)
    sa = torch.rand((7, K // 128), device="cuda")
    off = torch.zeros(E + 1, dtype=I32, device="cuda")
    off[1:] = 2
    off[E] = 7
    out = torch.empty((7, N), device="cuda")
    moe.moe_product_fp8(a, sa, b, sb, out, offsets=off)
    assert not out[:2].any()
    ref, bound = og.product(a[2:].view(torch.uint8).cpu().numpy(), sa[2:].cpu().numpy(), last.view(torch.uint8).cpu().numpy(),
                            sb[E - 1].cpu().numpy())
    assert (np.abs(f64(out[2:]) - ref) <= bound + EPS32 * (np.abs(ref) + bound)).all()


@pytest.mark.parametrize("tokens", [1, 64])
def test_example(tokens):
    """The block runs; its routing weights' gradient against differences of the routed part, which is
    linear in them."""
    block, x, residual = grouped_experts.make(gen.CONFIGS["tiny_ll_em"], tokens)
    out = block.forward(x, residual)
    assert out.isfinite().all()
    codes, scales, _ = ofp8.quantize_rows(f64(block.y.float()))
    assert (np.abs(scales / f64(block.scales) - 1) < 2.0 ** -7).all()     # the norm's own rows, from float32
    dout = torch.randn_like(out)
    dweights, dlogits = block.router_backward(dout)
    ref = torch.einsum("th,tkh->tk", dout.double(), block.experts.out.double()[block.position.long()])
    size = torch.einsum("th,tkh->tk", dout.double().abs(), block.experts.out.double()[block.position.long()].abs())
    assert ((dweights.double() - ref).abs() <= (block.y.shape[1] / 32 + 21) * EPS32 * size).all()
    routed = torch.empty((tokens, x.shape[1]), device="cuda")

    def loss(w):
        moe.moe_unsort_rows(block.experts.out, w, block.position, routed)
        return (routed.double() * dout.double()).sum(1)

    for j in range(block.weights.shape[1]):      # every token at once: a token's loss hangs on its own weights
        up, down = block.weights.clone(), block.weights.clone()
        up[:, j] += 1
        down[:, j] -= 1
        d = (loss(up) - loss(down)) / 2
        # two float32 sums over the picks, each a few roundings of terms of size |dout| |rows| |w|
        terms = (size * (block.weights.abs() + 1).double()).sum(1)
        assert ((d - dweights[:, j].double()).abs() <= 32 * EPS32 * terms + (block.y.shape[1] / 32 + 21) * EPS32 * size[:, j]).all()
    assert dlogits.isfinite().all()
