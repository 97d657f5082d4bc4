"""CPU oracle of the operators around the expert layer: residual addition with RMS norm, the
router, and the routed experts' FFN on 4-bit weights, in numpy float64 from their formulas.

TEST INFRASTRUCTURE ONLY (same rule as the rest of this package).  Nothing here is fast and
nothing is shared with the library.  Functions that name a bound return, beside the value,
how far a float32 evaluation may lie from it; the constants are worst cases of float32
rounding (2^-24 per operation) over the number of operations in a chain.
"""
import numpy as np

EPS32 = 2.0 ** -24
BF16 = 2.0 ** -8        # largest relative error of one rounding to bf16 (8-bit significand, to nearest)
E4M3 = 2.0 ** -4        # the same for an e4m3 code in its normal range
TC = 2.0 ** -14         # relative to sum |a b|: float32 sums on the tensor cores, K up to 2^14


# ---- residual addition and RMS norm ----------------------------------------------------------


def add_rmsnorm(x, res, w, eps):
    h = x if res is None else x + res
    rstd = 1.0 / np.sqrt((h * h).mean(1) + eps)
    return h, rstd, h * rstd[:, None] * w


def add_rmsnorm_backward(dout, h, w, rstd, dsum):
    """dx, dweight, and the float32 bounds of both.  A row's sum has at most 8 * 8 terms per
    thread and 37 more additions (five shuffles, 32 warps); a column's T / 304 per block and 64."""
    g = dout * w
    xhat = h * rstd[:, None]
    mean = (g * xhat).mean(1, keepdims=True)
    dx = rstd[:, None] * (g - xhat * mean)
    size = np.abs(rstd[:, None] * g) + np.abs(rstd[:, None] * xhat) * np.abs(g * xhat).mean(1, keepdims=True)
    if dsum is not None:
        dx = dx + dsum
        size = size + np.abs(dsum)
    terms = dout * xhat
    return dx, terms.sum(0), 110 * EPS32 * size, (len(h) / 304 + 72) * EPS32 * np.abs(terms).sum(0)


# ---- router ----------------------------------------------------------------------------------


def scores(logits, kind):
    """Scores of each expert; an absent one (logit -inf or NaN) has 0, +inf is the largest float."""
    l = np.where(np.isnan(logits), -np.inf, np.minimum(logits, np.finfo(np.float32).max))
    there = l > -np.inf
    if kind == "sigmoid":
        with np.errstate(over="ignore"):
            return np.where(there, 1.0 / (1.0 + np.exp(-np.where(there, l, 0.0))), 0.0), there
    top = np.where(there, l, -np.finfo(np.float64).max).max(1, keepdims=True)
    with np.errstate(over="ignore", under="ignore"):
        e = np.where(there, np.exp(np.where(there, l - top, 0.0)), 0.0)
    z = e.sum(1, keepdims=True)
    return np.where(z > 0, e / np.where(z > 0, z, 1.0), 0.0), there


def route(logits, bias, k, kind="softmax", groups=1, top_groups=1, pair=False, renorm=True, scale=1.0):
    """ids [T, k], weights [T, k] and, per token, the smallest gap above 0 between two computed
    keys (or group scores) whose order decides, relative to the largest key; infinite where
    the keys are the logits themselves, which are compared exactly."""
    T, E = logits.shape
    s, there = scores(logits, kind)
    by_logit = bias is None and (groups == 1 or not pair)
    key = np.minimum(logits, np.finfo(np.float32).max) if by_logit else s + (0.0 if bias is None else bias)
    if bias is not None:
        there = there & ~np.isnan(bias) & (bias > -np.inf)
    ids = np.full((T, k), -1, dtype=np.int64)
    w = np.zeros((T, k))
    gap = np.full(T, np.inf)
    size = E // groups
    for t in range(T):
        left = [e for e in range(E) if there[t, e]]
        big = max([abs(key[t, e]) for e in left] + [1e-300])
        if groups > 1:
            marks = []
            for g in range(groups):
                own = sorted((key[t, e] for e in left if e // size == g), reverse=True)
                marks.append(sum(own[:2]) if pair and own else own[0] if own else -np.inf)
            order = sorted(range(groups), key=lambda g: (-marks[g], g))
            if top_groups < groups and marks[order[top_groups]] > -np.inf:
                d = marks[order[top_groups - 1]] - marks[order[top_groups]]
                gap[t] = min(gap[t], d / big if d > 0 else np.inf)
            left = [e for e in left if e // size in order[:top_groups]]
        left.sort(key=lambda e: (-key[t, e], e))
        for a, b in zip(left[:k], left[1:k + 1]):
            d = key[t, a] - key[t, b]
            gap[t] = min(gap[t], d / big if d > 0 else np.inf)
        for j, e in enumerate(left[:k]):
            ids[t, j] = e
            w[t, j] = s[t, e]
    if by_logit:
        gap[:] = np.inf
    if renorm:
        z = w.sum(1, keepdims=True)
        w = np.where(z > 0, w / np.where(z > 0, z, 1.0), 0.0)
    return ids, w * scale, gap


def route_weights(logits, ids, kind, renorm, scale):
    """The weights of given picks: the function whose gradient route_backward is."""
    s, _ = scores(logits, kind)
    ok = ids >= 0
    p = np.take_along_axis(s, np.where(ok, ids, 0), 1) * ok
    if renorm:
        z = p.sum(1, keepdims=True)
        p = np.where(z > 0, p / np.where(z > 0, z, 1.0), 0.0)
    return p * scale


def route_backward(logits, ids, dw, kind, renorm, scale):
    """dlogits, and the float32 bound: 40 operations on a chain over the sizes of its terms."""
    s, _ = scores(logits, kind)
    T, k = ids.shape
    ok = ids >= 0
    at = np.where(ok, ids, 0)
    p = np.take_along_axis(s, at, 1) * ok
    g = np.where(ok, dw, 0.0) * scale
    size = np.abs(g)
    if renorm:
        z = p.sum(1, keepdims=True)
        z1 = np.where(z > 0, z, 1.0)
        size = np.where(ok & (z > 0), (size + (size * p).sum(1, keepdims=True) / z1) / z1, 0.0)
        g = np.where(ok & (z > 0), (g - (g * p).sum(1, keepdims=True) / z1) / z1, 0.0)
    d, m = np.zeros_like(s), np.zeros_like(s)
    for j in range(k):
        rows = np.nonzero(ok[:, j])[0]
        d[rows, ids[rows, j]] += g[rows, j]
        m[rows, ids[rows, j]] += size[rows, j]
    if kind == "sigmoid":   # 1 - s is the sigmoid of -logit, which cancels nothing
        return d * s * scores(-logits, kind)[0], 60 * EPS32 * m * s
    return s * (d - (d * s).sum(1, keepdims=True)), 60 * EPS32 * s * (m + (m * s).sum(1, keepdims=True))


# ---- 4-bit weights ----------------------------------------------------------------------------


def unpack_w4(codes, scales):
    """uint8 [..., K / 2], float scales [..., K / G] -> float64 [..., K]."""
    lo, hi = codes & 15, codes >> 4
    v = np.stack([lo, hi], -1).reshape(codes.shape[:-1] + (-1,)).astype(np.float64) - 8
    G = v.shape[-1] // scales.shape[-1]
    return v * np.repeat(scales.astype(np.float64), G, -1)


def forward_w4(x, ids, weights, w1, s1, w2, s2):
    """out [T, H] in float64, and the bound of a float32 evaluation that carries the activation
    as a bf16 pair (2^-16) and rounds out to bf16 once: the arithmetic of the bf16 layer on the
    weights that the codes stand for.  The 4-bit kernels carry the activation in f16 (2^-11), 32
    times as coarse; they meet this narrower bound in the tests too, which only a sum whose
    roundings all agreed would exceed."""
    T, H = x.shape
    I = w2.shape[2] * 2
    out, off = np.zeros((T, H)), np.zeros((T, H))
    for e in range(w1.shape[0]):
        picks = np.argwhere(ids == e)
        if not len(picks):
            continue
        up, down = unpack_w4(w1[e], s1[e]), unpack_w4(w2[e], s2[e])
        for t, j in picks:
            h, hs = up @ x[t], np.abs(up) @ np.abs(x[t])
            g, u = h[:I], h[I:]
            with np.errstate(over="ignore"):
                sg = g / (1 + np.exp(-g))
            act = sg * u
            # |silu'| <= 1.1; the product's error from either factor, the pair's rounding
            da = 1.1 * TC * hs[:I] * (np.abs(u) + TC * hs[I:]) + np.abs(sg) * TC * hs[I:] + 2.0 ** -16 * np.abs(act)
            out[t] += weights[t, j] * (down @ act)
            off[t] += abs(weights[t, j]) * (np.abs(down) @ (da + TC * np.abs(act)))
    return out, off + BF16 * np.abs(out) + 2.0 ** -133
