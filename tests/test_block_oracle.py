"""Pins of the block oracle: closed forms, library special cases, central differences."""
import numpy as np
import pytest
import torch

from oracle import block as ob

RNG = np.random.default_rng(11)


def test_norm_against_torch():
    x, r, w = RNG.normal(size=(5, 37)), RNG.normal(size=(5, 37)), RNG.normal(size=37)
    h, rstd, y = ob.add_rmsnorm(x, r, w, 1e-3)
    t = torch.nn.functional.rms_norm(torch.tensor(x + r), (37,), torch.tensor(w), 1e-3)
    np.testing.assert_allclose(y, t.numpy(), rtol=1e-12)
    np.testing.assert_allclose(h, x + r)


def test_norm_backward_against_autograd_and_differences():
    h, w, dout, ds = (RNG.normal(size=s) for s in ((4, 9), (9,), (4, 9), (4, 9)))
    th, tw = torch.tensor(h, requires_grad=True), torch.tensor(w, requires_grad=True)
    y = th * torch.rsqrt(th.square().mean(1, keepdim=True) + 0.1) * tw
    (y * torch.tensor(dout)).sum().backward()
    rstd = 1 / np.sqrt((h * h).mean(1) + 0.1)
    dx, dw, bx, bw = ob.add_rmsnorm_backward(dout, h, w, rstd, ds)
    np.testing.assert_allclose(dx, th.grad.numpy() + ds, rtol=1e-10)
    np.testing.assert_allclose(dw, tw.grad.numpy(), rtol=1e-10)
    assert (bx > 0).all() and (bw > 0).all()
    for i in range(9):
        d = np.zeros((4, 9))
        d[2, i] = 1e-6
        f = lambda v: (ob.add_rmsnorm(v, None, w, 0.1)[2] * dout).sum()  # noqa: E731
        assert abs((f(h + d) - f(h - d)) / 2e-6 - (dx - ds)[2, i]) < 1e-7


def test_route_by_hand():
    logits = np.log(np.array([[1.0, 4.0, 2.0, 3.0, 3.0, 1.0]]))      # softmax: 1 4 2 3 3 1 over 14
    ids, w, _ = ob.route(logits, None, 3, renorm=False)
    assert ids.tolist() == [[1, 3, 4]] and np.allclose(w, np.array([[4, 3, 3]]) / 14)
    ids, w, _ = ob.route(logits, None, 3, scale=2.0)
    assert np.allclose(w, [[0.8, 0.6, 0.6]])
    # groups (0 1) (2 3) (4 5): maxima 4 3 3, the tie goes to the second group
    assert ob.route(logits, None, 3, groups=3, top_groups=2)[0].tolist() == [[1, 3, 2]]
    # by pairs 5 5 4 over 14, then the bias lifts the last group to the top
    assert ob.route(logits, None, 2, groups=3, top_groups=2, pair=True)[0].tolist() == [[1, 3]]
    bias = np.array([0, 0, 0, 0, 0, 1.0])
    ids, w, _ = ob.route(logits, bias, 2, groups=3, top_groups=1, pair=True)
    assert ids.tolist() == [[5, 4]] and np.allclose(w, [[0.25, 0.75]])
    inf = np.inf
    ids, w, gap = ob.route(np.array([[-inf, np.nan, 2.0], [-inf] * 3]), None, 2)
    assert ids.tolist() == [[2, -1], [-1, -1]] and w.tolist() == [[1, 0], [0, 0]] and (gap == inf).all()
    assert np.allclose(ob.route(np.array([[inf, 1.0, inf]]), None, 2)[1], [[0.5, 0.5]])


@pytest.mark.parametrize("kind,renorm", [("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)])
def test_route_backward_against_differences(kind, renorm):
    l, c = RNG.normal(size=(3, 7)), RNG.normal(size=(3, 2))
    ids = ob.route(l, None, 2, kind)[0]
    ids[1, 1] = -1
    d, bound = ob.route_backward(l, ids, c, kind, renorm, 1.5)
    for t in range(3):
        for e in range(7):
            s = np.zeros_like(l)
            s[t, e] = 1e-6
            up, down = (ob.route_weights(l + v * s, ids, kind, renorm, 1.5) for v in (1, -1))
            assert abs(((up - down) * c).sum() / 2e-6 - d[t, e]) < 1e-8
    assert (bound >= 0).all()


def test_w4_by_hand_and_against_torch():
    assert ob.unpack_w4(np.array([[0x0f, 0x98]], np.uint8), np.array([[0.5, 2.0]])).tolist() == [[3.5, -4.0, 0.0, 2.0]]
    E, H, I, T = 2, 8, 6, 3
    w1, w2 = (RNG.integers(0, 256, s).astype(np.uint8) for s in ((E, 2 * I, H // 2), (E, H, I // 2)))
    s1, s2 = RNG.random((E, 2 * I, 2)), RNG.random((E, H, 3))
    x, ids, w = RNG.normal(size=(T, H)) * 0.1, np.array([[0, 1], [1, -1], [-1, -1]]), RNG.random((T, 2))
    out, bound = ob.forward_w4(x, ids, w, w1, s1, w2, s2)
    for t in range(T):
        ref = torch.zeros(H, dtype=torch.float64)
        for j, e in enumerate(ids[t]):
            if e >= 0:
                h = torch.tensor(ob.unpack_w4(w1[e], s1[e])) @ torch.tensor(x[t])
                ref += w[t, j] * torch.tensor(ob.unpack_w4(w2[e], s2[e])) @ (torch.nn.functional.silu(h[:I]) * h[I:])
        np.testing.assert_allclose(out[t], ref.numpy(), rtol=1e-10)
    assert (bound[0] > 0).all() and (out[2] == 0).all()
    # a planted mistake (gate and up exchanged) lies far outside the bound
    swapped = ob.forward_w4(x, ids, w, np.roll(w1, I, 1), np.roll(s1, I, 1), w2, s2)[0]
    assert (np.abs(swapped - out)[0] > bound[0]).any()
