"""4-bit quantisation of weights that are not finite: none of them becomes a number."""
import os

import pytest
import torch

import combine_topk_ids_gb300 as moe

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    if not os.path.exists(moe.LIB_PATH):
        moe.build()


def quantize(w, G):
    codes = torch.empty(w.shape[:-1] + (w.shape[-1] // 2,), dtype=torch.uint8, device="cuda")
    scales = torch.empty(w.shape[:-1] + (w.shape[-1] // G,), dtype=BF, device="cuda")
    moe.moe_quantize_w4(w, G, codes, scales)
    return codes, scales


@pytest.mark.parametrize("G", [32, 64, 128])
@pytest.mark.parametrize("value", [NAN, INF, -INF])
@pytest.mark.parametrize("at", [0, 1, 17, 31])
def test_groups_with_a_value_that_is_not_finite(G, value, at):
    w = (torch.randn((5, 256), generator=torch.Generator().manual_seed(1)) * 0.05).to(BF).cuda()
    codes, scales = quantize(w, G)
    bad = w.clone()
    bad[2, 128 + at] = value
    c, s = quantize(bad, G)
    group = 128 // G
    assert s[2, group].isnan() and (c[2, 64:64 + G // 2] == 0x88).all()
    keep = torch.ones_like(s, dtype=torch.bool)
    keep[2, group] = False
    assert torch.equal(s[keep], scales[keep])
    assert torch.equal(c.view(5, 256 // G, -1)[keep], codes.view(5, 256 // G, -1)[keep])


def test_such_a_weight_shows_in_the_output():
    """In the columns of its row alone, for the tokens that go to its expert."""
    H, E, k, I = 256, 4, 1, 128
    g = torch.Generator().manual_seed(2)
    w1, w2 = ((torch.randn(s, generator=g) * 0.05).to(BF).cuda() for s in ((E, 2 * I, H), (E, H, I)))
    w2[1, 77, 5] = NAN
    layer = moe.MoELayerW4(4, H, E, k, I, 64)
    layer.quantize_weights(w1, w2)
    x = torch.randn((4, H), generator=g).to(BF).cuda()
    out = layer.forward(x, torch.tensor([[0], [1], [2], [1]], device="cuda"), torch.ones((4, 1), device="cuda"))
    nan = out.isnan()
    assert nan[[1, 3], 77].all() and nan.sum() == 2
