"""The gradient of sigmoid scores at confident experts: its slope s (1 - s) is tiny there, and
1 - s holds none of its digits once s is rounded."""
import os

import numpy as np
import pytest
import torch

import combine_topk_ids_gb300 as moe

pytestmark = pytest.mark.gpu
EPS32 = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    if not os.path.exists(moe.LIB_PATH):
        moe.build()


@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("E", [8, 100, 256])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_sigmoid_gradient_of_confident_experts(E, renorm, dtype):
    """Logits of either sign and up to 30 in size, relative to the slope itself.  Bound: a score's
    and its complement's relative errors are at most (|logit| + 16) 2^-23 each, where
    renormalised two more of them, and a dozen roundings."""
    T, k, scale = 12, 4, 1.5
    rng = np.random.default_rng(4)
    size = np.array([8.0, 10, 12, 14, 15, 16, 17, 18, 20, 24, 28, 30])[:, None]
    l = torch.tensor((rng.random((T, E)) * 0.2 + 0.8) * size * rng.choice([-1.0, 1.0], (T, E))).to(dtype).cuda()
    ids = torch.tensor(rng.permuted(np.tile(np.arange(E), (T, 1)), axis=1)[:, :k].copy()).cuda()
    dw = torch.tensor(rng.normal(size=(T, k)), dtype=torch.float32, device="cuda")
    got = torch.empty_like(l)
    moe.moe_route_topk_backward(moe.make_router(E, k, "sigmoid", renormalize=renorm, scale=scale), l, ids, dw, got)
    at, g = ids.cpu().numpy(), dw.cpu().double().numpy() * scale
    lp = np.take_along_axis(l.cpu().double().numpy(), at, 1)
    s, slope = 1 / (1 + np.exp(-lp)), 1 / (1 + np.exp(lp))
    q, along, along_size = s, 0.0, 0.0
    if renorm:
        q = s / s.sum(1, keepdims=True)
        along, along_size = (g * q).sum(1, keepdims=True), (np.abs(g) * q).sum(1, keepdims=True)
    pick, reach = q * slope * (g - along), q * slope * (np.abs(g) + along_size)
    bound = (2 * (4 if renorm else 2) * (np.abs(lp).max(1, keepdims=True) + 16) + 12) * EPS32 * reach
    if dtype == torch.bfloat16:
        bound = bound + 2.0 ** -8 * np.abs(pick)
    out = got.cpu().double().numpy()
    d = np.abs(np.take_along_axis(out, at, 1) - pick)
    assert (d <= bound + 1e-37).all(), (d / reach).max(1)
    np.put_along_axis(out, at, 0.0, 1)
    assert (out == 0).all()

