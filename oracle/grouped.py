"""CPU oracle of the operators on expert-grouped rows: the order of a batch's picks, rows in it
and back, SwiGLU in front of a quantisation, and the block-scaled FP8 product, in numpy float64
from their formulas.

TEST INFRASTRUCTURE ONLY (same rule as the rest of this package).  Functions that name a bound
return, beside the value, how far a float32 evaluation may lie from it: worst cases of float32
rounding (2^-24 per operation, 2^-23 where a unit may cut digits off) over the number of
operations in a chain.
"""
import numpy as np

from .block import EPS32
from .fp8 import decode_e4m3


def order(ids, E):
    """offsets [E + 1], position [T, k] and source [T k], pick by pick in (expert, token, pick) order."""
    flat = ids.reshape(-1)
    position, source = np.full(flat.shape, -1, np.int64), np.full(flat.shape, -1, np.int64)
    offsets, r = np.zeros(E + 1, np.int64), 0
    by_expert = [[] for _ in range(E)]
    for i, e in enumerate(flat):
        if 0 <= e < E:
            by_expert[e].append(i)
    for e in range(E):
        for i in by_expert[e]:
            position[i], source[r], r = r, i, r + 1
        offsets[e + 1] = r
    return offsets, position.reshape(ids.shape), source


def sort_rows(x, position, rows):
    """rows with x[t] at every pick's position."""
    rows = rows.copy()
    for t, p in enumerate(position):
        for r in p:
            if 0 <= r < len(rows):
                rows[r] = x[t]
    return rows


def unsort_rows(rows, weights, position):
    """out and its float32 bound: a product and an addition for each pick."""
    T, k = position.shape
    out, size = np.zeros((T, rows.shape[1])), np.zeros((T, rows.shape[1]))
    for t in range(T):
        for j in range(k):
            if 0 <= position[t, j] < len(rows):
                term = (1.0 if weights is None else weights[t, j]) * rows[position[t, j]]
                out[t] += term
                size[t] += np.abs(term)
    return out, 2 * k * EPS32 * size


def unsort_rows_backward(dout, rows, weights, position, drows):
    """drows (with every pick's row replaced), dweights and its float32 bound.  A dot product is
    spread over 32 threads at least, 8 columns at a time, and has 13 more additions."""
    drows, T, k = drows.copy(), *position.shape
    dw, size = np.zeros((T, k)), np.zeros((T, k))
    for t in range(T):
        for j in range(k):
            p = position[t, j]
            if 0 <= p < len(drows):
                drows[p] = (1.0 if weights is None else weights[t, j]) * dout[t]
                if rows is not None:
                    dw[t, j] = (dout[t] * rows[p]).sum()
                    size[t, j] = np.abs(dout[t] * rows[p]).sum()
    chain = rows.shape[1] / 32 + 8 + 13 if rows is not None else 0
    return drows, dw, chain * EPS32 * size


def swiglu(gate_up):
    """silu(gate) * up, and the relative bound of its float32 evaluation: the power of two (2 steps of
    2^-23), its correction and the sum (1), the reciprocal (1) and two products (1), and 3 to spare."""
    I = gate_up.shape[1] // 2
    g, u = gate_up[:, :I], gate_up[:, I:]
    with np.errstate(over="ignore"):
        return g / (1 + np.exp(-g)) * u, 8 * 2.0 ** -23


def product(a, sa, b, sb):
    """The product of codes a [M, K] and b [N, K] (uint8) with their scales, and its float32 bound.
    Sums of 128 in the tensor cores may cut digits at each addition; two products and an addition
    of 2^-24 each for a block's scales, and three more additions across a cluster."""
    da = decode_e4m3(a) * np.repeat(sa.astype(np.float64), 128, 1)
    db = decode_e4m3(b) * np.repeat(np.repeat(sb.astype(np.float64), 128, 0)[:len(b)], 128, 1)
    chain = 128 * 2.0 ** -23 + (a.shape[1] // 128 + 2 + 3) * EPS32
    return da @ db.T, chain * (np.abs(da) @ np.abs(db).T)
