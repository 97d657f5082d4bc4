"""The router's gradient where scores are tiny, against its formula in 64 bits:

    sigmoid, renormalised   q (1 - s) (g - sum g q)      softmax, renormalised   q (g - sum g q)

with s the picks' scores, q = s / sum s (0 where the float32 scores' sum is 0) and
g = scale * dweights; 0 outside the picks.
"""
import os

import numpy as np
import pytest
import torch

import combine_topk_ids_gb300 as moe

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
EPS32 = 2.0 ** -24
LOW = torch.finfo(F32).min


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    if not os.path.exists(moe.LIB_PATH):
        moe.build()


def backward(logits, ids, dweights, kind, renorm, scale, dtype=F32):
    l = torch.tensor(logits, dtype=torch.float64).to(dtype).cuda()
    i, g = torch.tensor(ids, device="cuda"), torch.tensor(dweights, dtype=F32, device="cuda")
    out = torch.full(l.shape, 77.0, dtype=dtype, device="cuda")
    moe.moe_route_topk_backward(moe.make_router(l.shape[1], i.shape[1], kind, renormalize=renorm, scale=scale),
                                l, i, g, out)
    return l.cpu().double().numpy(), out.cpu().double().numpy()


def renormalised(logits, ids, dweights, kind, scale):
    """The formula (ids distinct, all there), and the bound of a float32 evaluation: a score's
    relative error is at most (|logit| + 16) 2^-23 (the exponent's rounding, the hardware's power
    of two and reciprocal), and a result takes four of them and a dozen roundings."""
    l = np.take_along_axis(logits, ids, 1)
    if kind == "sigmoid":
        s, slope = 1 / (1 + np.exp(-l)), 1 / (1 + np.exp(l))
        far = np.abs(l).max(1, keepdims=True)
    else:
        top = logits.max(1, keepdims=True)
        s, slope = np.exp(l - top), np.ones_like(l)
        far = (top - l).max(1, keepdims=True)
    q = s / s.sum(1, keepdims=True)
    g = np.asarray(dweights) * scale
    pick = q * slope * (g - (g * q).sum(1, keepdims=True))
    size = q * slope * (np.abs(g) + (np.abs(g) * q).sum(1, keepdims=True))
    ref, bound = np.zeros(logits.shape), np.zeros(logits.shape)
    np.put_along_axis(ref, ids, pick, 1)
    np.put_along_axis(bound, ids, (8 * (far + 16) + 12) * EPS32 * size, 1)
    return ref, bound + 1e-37


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("E", [8, 40, 256])
def test_no_score_left_sigmoid(E, dtype):
    """Every expert of a token at the type's lowest value: the weights are 0 whatever the logits,
    and so is the gradient, for weight gradients of any size."""
    logits = np.full((3, E), float(torch.finfo(dtype).min))
    logits[1] = np.random.default_rng(0).normal(size=E)
    ids = np.tile(np.arange(4), (3, 1))
    dw = np.array([[10.0, -7, 1.5, 0.1]] * 2 + [[1e4, -1e4, 3e30, 5]])
    _, got = backward(logits, ids, dw, "sigmoid", True, 2.5, dtype)
    assert (got[0] == 0).all() and (got[2] == 0).all()
    assert np.isfinite(got[1]).all() and (got[1, :4] != 0).all()


@pytest.mark.parametrize("E", [8, 40, 256])
def test_no_score_left_softmax(E):
    """Picks that a bias has moved to experts without a score: 0 over the whole row."""
    logits = np.full((2, E), LOW)
    logits[:, 0] = 1.0
    ids = np.array([[1, 2, 3], [0, 1, 2]])
    _, got = backward(logits, ids, [[10.0, -7, 3]] * 2, "softmax", True, 2.5)
    assert (got == 0).all()      # the second row's weights are 1, 0, 0 and stay so


@pytest.mark.parametrize("kind", ["sigmoid", "softmax"])
@pytest.mark.parametrize("E", [8, 256])
def test_smallest_scores(kind, E):
    """Scores just above float32's smallest normal number, with large weight gradients."""
    rng = np.random.default_rng(1)
    logits = rng.normal(size=(5, E)) - (0.0 if kind == "softmax" else 60.0)
    logits[:, 0] = 0.0 if kind == "softmax" else -60.0
    at = np.array([[1, 2, 3, 5]] * 5)
    np.put_along_axis(logits, at, -86.0 + rng.random((5, 4)) * np.array([[0.0], [0.5], [3], [20], [60]]), 1)
    if kind == "softmax":
        logits[logits > 0] = 0.0
    logits = np.float32(logits).astype(np.float64)
    dw = rng.normal(size=(5, 4)) * np.array([[10.0], [1e3], [10], [1], [1e6]])
    dw = np.float32(dw).astype(np.float64)
    _, got = backward(logits, at, dw, kind, True, 2.5)
    ref, bound = renormalised(logits, at, dw, kind, 2.5)
    assert (np.abs(got - ref) <= bound).all(), np.abs(got - ref).max()


@pytest.mark.parametrize("kind", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [True, False])
def test_picks_that_take_no_part(kind, renorm):
    """Ids that are none and experts that are absent: whatever their weights' gradients hold."""
    inf, nan = float("inf"), float("nan")
    logits = np.array([[0.5, -inf, nan, 1.0, -1.0, 0.0, 2.0, 0.25]] * 2)
    ids = np.array([[0, 1, 2, 3], [0, -1, 8, 3]])
    dw = np.array([[1.0, nan, inf, -2.0], [1.0, nan, inf, -2.0]])
    _, got = backward(logits, ids, dw, kind, renorm, 1.0)
    assert np.isfinite(got).all() and (got[0] == got[1]).all() and (got[:, 0] != 0).all()
    assert (got[:, 1:3] == 0).all()
