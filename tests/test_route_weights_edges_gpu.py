"""The router's weights where the picked scores are tiny."""
import os

import numpy as np
import pytest
import torch

import combine_topk_ids_gb300 as moe
from oracle import block as ob

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    if not os.path.exists(moe.LIB_PATH):
        moe.build()


def route(logits, bias, k, **rule):
    l, b = (torch.tensor(v, dtype=torch.float32, device="cuda") for v in (logits, bias))
    ids = torch.empty((l.shape[0], k), dtype=torch.int64, device="cuda")
    w = torch.empty((l.shape[0], k), device="cuda")
    moe.moe_route_topk(moe.make_router(l.shape[1], k, **rule), l, b, ids, w)
    return ids.cpu().numpy(), w.cpu().double().numpy()


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E", [16, 256, 2048])
def test_renormalised_weights_of_tiny_scores(kind, E):
    """A bias has moved the picks to experts whose scores lie at float32's smallest normal numbers
    (the other experts share the softmax's sum): their weights still add up to the scale.
    Bound: a score's relative error is at most (|logit| + 16) 2^-23, a weight's twice that."""
    k, scale = 8, 2.5
    logits = np.zeros((4, E))
    logits[:, :k] = np.float32(-86.5 + np.random.default_rng(2).random((4, k)) * np.array([[0.0], [0.1], [2], [30]]))
    if kind == "sigmoid":
        logits[:, k:] = -70.0
    bias = np.zeros(E)
    bias[:k] = np.arange(k, 0, -1)
    ids, w = route(logits, bias, k, score=kind, renormalize=True, scale=scale)
    ref_ids, ref, gap = ob.route(logits, bias, k, kind, scale=scale)
    assert (gap > 2e-6).all()
    np.testing.assert_array_equal(ids, ref_ids)
    assert (np.abs(w - ref) <= 2 * (86.5 + 16) * 2.0 ** -23 * ref).all(), (w, ref)
    np.testing.assert_allclose(w.sum(1), scale, rtol=1e-5)
