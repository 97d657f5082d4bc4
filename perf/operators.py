"""The measured cases of the operators around the expert layer.

norm    the residual's addition and RMS norm in front of the layer (bf16 rows, and e4m3
        codes with one scale per 128 columns), and its gradient
route   the router: expert ids and weights from the gate's logits, and its gradient
w4      the routed experts' SwiGLU FFN of a decode batch with 4-bit weights and group scales

With `own` false, run() computes the plain form with elementary torch operations in 32
bits; with `own` true it calls combine_topk_ids_gb300.
"""
import math

import torch

own = False

EPS = 1e-6


def listed():
    return [
        # one token of the 7168-wide decode: a norm between two layers, all latency
        norm("norm_one_token", 1, 7168, out="both"),
        # the default workload's prefill batch (8 x 4096 tokens) on its way to the FP8 dispatch
        # and the gate
        norm("norm_prefill_fp8", 32768, 7168, out="both"),
        # rows whose length leaves all but the first off a 16-byte boundary, a ragged token count
        norm("norm_odd_rows", 4999, 2047, out="bf16", weight="fp32"),
        # a training step's gradient at the 4096-wide model
        norm("norm_backward", 8192, 4096, back=True),
        # the decode batch of the 256-expert model: sigmoid scores, balance bias, 4 of 8 groups
        route("route_decode", 64, 256, 8, score="sigmoid", bias=True, groups=8, kept=4, pair=True, scale=2.5),
        # the same router over the prefill batch
        route("route_prefill", 32768, 256, 8, score="sigmoid", bias=True, groups=8, kept=4, pair=True, scale=2.5),
        # the ragged workload's 128 experts, softmax over bf16 logits with equal values among
        # them, some experts switched off and some tokens with no expert left
        route("route_softmax_masked", 16381, 128, 4, score="softmax", logits="bf16", masked=True),
        # the gradient of the prefill batch's routing weights, scores not renormalised
        route("route_backward", 32768, 256, 8, score="softmax", renorm=False, back=True),
        # the smallest call: three tokens of the smallest model, one pick in four masked
        w4("w4_tiny", 3, 256, 8, 2, 512, 32, drop=0.25),
        # one token of the 256-expert model
        w4("w4_one_token", 1, 7168, 256, 8, 2048, 128),
        # 16 tokens over 8 wide experts: about four rows for each expert
        w4("w4_wide_experts", 16, 4096, 8, 2, 14336, 64),
        # 64 tokens of the 256-expert model: nearly every expert is read
        w4("w4_batch", 64, 7168, 256, 8, 2048, 128),
    ]


def norm(name, tokens, hidden, out="bf16", residual=True, weight="bf16", back=False):
    return {"name": name, "op": "norm", "back": back, "tokens": tokens, "hidden": hidden, "out": out,
            "residual": residual, "weight": weight}


def route(name, tokens, experts, k, score, bias=False, groups=1, kept=1, pair=False, renorm=True, scale=1.0,
          logits="fp32", masked=False, back=False):
    return {"name": name, "op": "route", "back": back, "tokens": tokens, "experts": experts, "k": k,
            "score": score, "bias": bias, "groups": groups, "kept": kept, "pair": pair, "renorm": renorm,
            "scale": scale, "logits": logits, "masked": masked}


def w4(name, tokens, hidden, experts, k, inter, group, drop=0.0):
    return {"name": name, "op": "w4", "tokens": tokens, "hidden": hidden, "experts": experts, "k": k,
            "inter": inter, "group": group, "drop": drop}


def draw(rng):
    def spread(lo, hi):   # even over the logarithm
        n = 0
        while not lo <= n <= hi or n == 3072:
            n = round(math.exp(rng.uniform(math.log(lo), math.log(hi))))
        return n

    def of128(lo, hi):
        n = 0
        while not n or n == 3072:
            n = 128 * max(1, round(spread(lo, hi) / 128))
        return n

    op = rng.choice(("norm", "route", "w4"))
    while True:
        if op == "norm":
            back, out = rng.random() < 0.4, rng.choice(("bf16", "fp8", "both"))
            out = "bf16" if back else out
            hidden = of128(128, 8192) if out != "bf16" or rng.random() < 0.5 else spread(32, 8192)
            case = norm("", spread(1, 32768), hidden, out, rng.random() < 0.75,
                        rng.choice(("bf16", "fp32")), back)
            fits = case["tokens"] * hidden <= 32768 * 7168
        elif op == "route":
            experts = rng.choice((8, 16, 60, 64, 72, 128, 160, 256, 384, 512)) if rng.random() < 0.7 else spread(4, 2048)
            groups = rng.choice([g for g in (1, 2, 4, 8, 16) if experts % g == 0])
            kept = rng.randint(max(1, groups // 2), groups)
            k = rng.randint(1, min(16, experts // groups * kept))
            case = route("", spread(1, 32768), experts, k, rng.choice(("softmax", "sigmoid")), rng.random() < 0.5,
                         groups, kept, rng.random() < 0.5, rng.random() < 0.6, rng.choice((1.0, 2.5)),
                         rng.choice(("fp32", "bf16")), rng.random() < 0.3, rng.random() < 0.35)
            fits = case["tokens"] * experts <= 32768 * 256
        else:
            experts = rng.choice((4, 8, 16, 32, 60, 64, 128, 160, 256))
            case = w4("", spread(1, 64), of128(128, 7168), experts, rng.randint(1, min(8, experts)),
                      of128(128, 14336), rng.choice((32, 64, 128)), rng.choice((0.0, 0.0, 0.2)))
            fits = experts * case["hidden"] * case["inter"] <= 256 * 7168 * 2048
        if fits:
            del case["name"]
            return case


# ---- inputs ----------------------------------------------------------------------------------


def generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def inputs(case, seed):
    """The operator's inputs alone, made on the GPU from the seed."""
    return {"norm": norm_inputs, "route": route_inputs, "w4": w4_inputs}[case["op"]](case, generator(seed))


def norm_inputs(c, g):
    T, H = c["tokens"], c["hidden"]

    def rows(scale):
        return torch.randn((T, H), generator=g, device="cuda", dtype=torch.bfloat16).mul_(scale)

    # a residual stream a few times as large as what a block adds, tokens of different size
    size = torch.rand((T, 1), generator=g, device="cuda").mul_(2).exp_().to(torch.bfloat16)
    i = {"weight": torch.randn(H, generator=g, device="cuda").mul_(0.2).add_(1)}
    if c["weight"] == "bf16":
        i["weight"] = i["weight"].bfloat16()
    if c["back"]:
        i["h"] = rows(1).mul_(size)
        i["rstd"] = torch.rsqrt(i["h"].float().square().mean(1) + EPS)
        i["dout"] = rows(0.01)
        i["dsum"] = rows(0.01) if c["residual"] else None
    else:
        i["x"] = rows(1)
        i["residual"] = rows(3).mul_(size) if c["residual"] else None
    return i


def route_inputs(c, g):
    T, E, k = c["tokens"], c["experts"], c["k"]
    lean = torch.randn(E, generator=g, device="cuda").mul_(0.5)   # experts are not equally liked
    bias = torch.randn(E, generator=g, device="cuda").mul_(0.05 if c["score"] == "sigmoid" else 0.2 / E) if c["bias"] else None
    off = torch.rand(E, generator=g, device="cuda") < 0.06 if c["masked"] else None
    if off is not None:
        off[0] = False
    none = torch.rand(T, generator=g, device="cuda") < 0.01 if c["masked"] else None

    def some(n):
        v = torch.randn((n, E), generator=g, device="cuda").add_(lean)
        v = v.bfloat16() if c["logits"] == "bf16" else v
        return v if off is None else v.masked_fill_(off, -math.inf)

    logits = some(T)
    if none is not None:
        logits[none] = -math.inf
    # Where two keys at a place that decides lie nearer than 32-bit scores resolve, any order is
    # right: such tokens are drawn again, so that every case has one answer.  Equal keys stay.
    if by_score(c):
        for _ in range(40):
            bad = unclear(c, logits, bias).nonzero().flatten()
            if not len(bad):
                break
            logits[bad] = some(len(bad))
    i = {"logits": logits, "bias": bias}
    if c["back"]:
        i["ids"] = route_plain(c, i)["ids"]
        i["dweights"] = torch.randn((T, k), generator=g, device="cuda")
    return i


def by_score(c):
    """Whether the experts' order hangs on computed scores, and not on the logits alone."""
    return c["bias"] or (c["groups"] > 1 and c["pair"])


def unclear(c, logits, bias):
    E, n = c["experts"], c["groups"]
    l = logits.double()
    s = l.softmax(1).nan_to_num(0.0) if c["score"] == "softmax" else l.sigmoid()
    key = (s if bias is None else s + bias.double()).masked_fill(l == -math.inf, -math.inf)
    limit = 2e-6 * key.masked_fill(key == -math.inf, 0).abs().amax(1, keepdim=True)

    def near(a):
        d = a[:, :-1] - a[:, 1:]
        return ((d > 0) & (d < limit)).any(1)

    bad = torch.zeros(len(l), dtype=torch.bool, device=l.device)
    if n > 1:
        top = key.view(-1, n, E // n).sort(2, descending=True)[0]
        score = top[:, :, 0]
        if c["pair"] and E // n > 1:
            score = score + top[:, :, 1].masked_fill(top[:, :, 1] == -math.inf, 0)
        score, order = score.sort(dim=1, descending=True, stable=True)
        if c["kept"] < n:
            bad |= near(score[:, c["kept"] - 1:c["kept"] + 1])
        keep = torch.zeros((len(l), n), dtype=torch.bool, device=l.device).scatter_(1, order[:, :c["kept"]], True)
        key = key.masked_fill(~keep.repeat_interleave(E // n, 1), -math.inf)
    return bad | near(key.sort(1, descending=True)[0][:, :c["k"] + 1])


def w4_inputs(c, g):
    T, H, E, k, I, G = (c[n] for n in ("tokens", "hidden", "experts", "k", "inter", "group"))

    def codes(*shape):
        return torch.randint(0, 256, shape, generator=g, device="cuda", dtype=torch.uint8)

    def scales(rows, cols, size):
        return torch.rand((E, rows, cols // G), generator=g, device="cuda").add_(0.5).mul_(size).bfloat16()

    ids = torch.rand((T, E), generator=g, device="cuda").argsort(1)[:, :k].contiguous()
    ids[torch.rand((T, k), generator=g, device="cuda") < c["drop"]] = -1
    w = torch.rand((T, k), generator=g, device="cuda").add_(0.05)
    return {"x": torch.randn((T, H), generator=g, device="cuda", dtype=torch.bfloat16), "ids": ids,
            "weights": w / w.sum(1, keepdim=True),
            "w1": codes(E, 2 * I, H // 2), "s1": scales(2 * I, H, 0.25 / math.sqrt(H)),
            "w2": codes(E, H, I // 2), "s2": scales(H, I, 0.5 / math.sqrt(I))}


def prepare(case, seed):
    s = {"case": case, **inputs(case, seed)}
    if not own:
        return s
    import combine_topk_ids_gb300 as moe

    s["moe"] = moe

    def empty(*shape, dtype=torch.float32):
        return torch.empty(shape, dtype=dtype, device="cuda")

    T = case["tokens"]
    if case["op"] == "norm":
        H = case["hidden"]
        if case["back"]:
            s["dx"], s["dweight"] = empty(T, H, dtype=torch.bfloat16), empty(H)
            s["workspace"] = empty(moe.moe_add_rmsnorm_workspace_size(T, H), dtype=torch.uint8)
        else:
            s["sum"] = empty(T, H, dtype=torch.bfloat16) if case["residual"] else None
            s["out"] = empty(T, H, dtype=torch.bfloat16) if case["out"] != "fp8" else None
            s["codes"] = empty(T, H, dtype=torch.float8_e4m3fn) if case["out"] != "bf16" else None
            s["scales"] = empty(T, H // 128) if case["out"] != "bf16" else None
            s["rstd"] = empty(T)
    elif case["op"] == "route":
        E, k = case["experts"], case["k"]
        s["router"] = moe.make_router(E, k, score=case["score"], groups=case["groups"], top_groups=case["kept"],
                                      group_score="top2" if case["pair"] else "max", renormalize=case["renorm"],
                                      scale=case["scale"])
        if case["back"]:
            s["dlogits"] = torch.empty_like(s["logits"])
        else:
            s["ids"], s["weights"] = empty(T, k, dtype=torch.int64), empty(T, k)
    else:
        s["layer"] = moe.MoELayerW4(T, case["hidden"], case["experts"], case["k"], case["inter"], case["group"])
        s["layer"].set_weights(*(s.pop(n) for n in ("w1", "s1", "w2", "s2")))
    return s


# ---- one pass --------------------------------------------------------------------------------


def run(s):
    c = s["case"]
    if c["op"] == "norm":
        return (norm_back if c["back"] else norm_run)(s)
    if c["op"] == "route":
        return (route_back if c["back"] else route_run)(s)
    return s["layer"].forward(s["x"], s["ids"], s["weights"]) if own else w4_plain(s)


def norm_run(s):
    if own:
        s["moe"].moe_add_rmsnorm(s["x"], s["residual"], s["weight"], EPS, sum_out=s["sum"], out=s["out"],
                                 out_fp8=s["codes"], scales=s["scales"], rstd=s["rstd"])
        return {n: s[n] for n in ("sum", "out", "codes", "scales", "rstd")}
    h = s["x"].float()
    if s["residual"] is not None:
        h = h + s["residual"]
    rstd = 1 / (h.square().mean(1) + EPS).sqrt()
    y = h * rstd[:, None] * s["weight"]
    r = {"sum": h.bfloat16() if s["residual"] is not None else None, "rstd": rstd}
    if s["case"]["out"] != "fp8":
        r["out"] = y.bfloat16()
    if s["case"]["out"] != "bf16":
        y = y.view(len(y), -1, 128)
        a = y.abs().amax(2).clamp_min(2.0 ** -100)
        r["codes"] = (y * (448 / a)[:, :, None]).view(h.shape).to(torch.float8_e4m3fn)
        r["scales"] = a / 448
    return r


def norm_back(s):
    if own:
        s["moe"].moe_add_rmsnorm_backward(s["dout"], s["h"], s["weight"], s["rstd"], s["dx"], s["dweight"],
                                          s["workspace"], dsum=s["dsum"])
        return {"dx": s["dx"], "dweight": s["dweight"]}
    rstd = s["rstd"][:, None]
    xhat = s["h"] * rstd
    dout = s["dout"].float()
    g = dout * s["weight"]
    dx = rstd * (g - xhat * (g * xhat).mean(1, keepdim=True))
    if s["dsum"] is not None:
        dx = dx + s["dsum"]
    return {"dx": dx.bfloat16(), "dweight": (dout * xhat).sum(0)}


def route_run(s):
    if own:
        s["moe"].moe_route_topk(s["router"], s["logits"], s["bias"], s["ids"], s["weights"])
        return {"ids": s["ids"], "weights": s["weights"]}
    return route_plain(s["case"], s)


def scores(c, logits):
    """The experts' scores in 32 bits; an expert whose logit is -inf has none (0)."""
    if c["score"] == "sigmoid":
        return 1 / (1 + torch.exp(-logits))
    p = torch.exp(logits - logits.amax(1, keepdim=True).clamp_min(-3e38))
    return p / p.sum(1, keepdim=True).clamp_min(1e-38)


def route_plain(c, s):
    E, n = c["experts"], c["groups"]
    logits = s["logits"].float()
    score = scores(c, logits)
    key = logits
    if by_score(c):
        key = score if s["bias"] is None else score + s["bias"]
        key = key.masked_fill(logits == -math.inf, -math.inf)
    if n > 1:
        top = key.view(-1, n, E // n).sort(2, descending=True)[0]
        group = top[:, :, 0]
        if c["pair"] and E // n > 1:
            group = group + top[:, :, 1].masked_fill(top[:, :, 1] == -math.inf, 0)
        best = group.sort(dim=1, descending=True, stable=True)[1][:, :c["kept"]]
        keep = torch.zeros_like(group, dtype=torch.bool).scatter_(1, best, True)
        key = key.masked_fill(~keep.repeat_interleave(E // n, 1), -math.inf)
    key, ids = key.sort(dim=1, descending=True, stable=True)
    key, ids = key[:, :c["k"]], ids[:, :c["k"]]
    w = score.gather(1, ids).masked_fill(key == -math.inf, 0)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True).clamp_min(1e-38)
    return {"ids": ids.masked_fill(key == -math.inf, -1), "weights": w * c["scale"]}


def route_back(s):
    c = s["case"]
    if own:
        s["moe"].moe_route_topk_backward(s["router"], s["logits"], s["ids"], s["dweights"], s["dlogits"])
        return s["dlogits"]
    score = scores(c, s["logits"].float())
    there = s["ids"] >= 0
    at = s["ids"].clamp_min(0)
    p = score.gather(1, at) * there
    g = s["dweights"] * c["scale"] * there
    if c["renorm"]:
        z = p.sum(1, keepdim=True).clamp_min(1e-38)
        g = (g - (g * p).sum(1, keepdim=True) / z) / z * there
    ds = torch.zeros_like(score).scatter_add_(1, at, g)
    if c["score"] == "sigmoid":
        d = ds * score * (1 - score)
    else:
        d = score * (ds - (ds * score).sum(1, keepdim=True))
    return d.to(s["logits"].dtype)


def unpack(codes, scales):
    """[.., rows, cols / 2] codes and [.., rows, cols / G] scales -> the weights in 32 bits."""
    v = torch.stack((codes & 15, codes >> 4), -1).view(*scales.shape, -1).float().sub_(8).mul_(scales[..., None])
    return v.view(*codes.shape[:-1], -1)


def w4_plain(s):
    c = s["case"]
    T, k, E, I = c["tokens"], c["k"], c["experts"], c["inter"]
    x, ids = s["x"].float(), s["ids"]
    w = s["weights"] * (ids >= 0)
    if T * k < E:   # the picked experts alone, pick by pick
        e = ids.clamp_min(0).flatten()
        x = x.repeat_interleave(k, 0)[:, :, None]
        gate, up = (unpack(s["w1"][e], s["s1"][e]) @ x).split(I, 1)
        y = unpack(s["w2"][e], s["s2"][e]) @ (gate / (1 + torch.exp(-gate)) * up)
        return (y.view(T, k, -1) * w[:, :, None]).sum(1).bfloat16()
    gate, up = (x @ unpack(s["w1"], s["s1"]).mT).split(I, 2)   # every expert on every token
    y = (gate / (1 + torch.exp(-gate)) * up) @ unpack(s["w2"], s["s2"]).mT
    share = torch.zeros((T, E), device=x.device).scatter_add_(1, ids.clamp_min(0), w)
    return (y * share.T[:, :, None]).sum(0).bfloat16()


# ---- what a pass cannot do without -----------------------------------------------------------


def work(case):
    T = case["tokens"]
    if case["op"] == "norm":
        n, H = T * case["hidden"], case["hidden"]
        weight = H * (2 if case["weight"] == "bf16" else 4)
        if case["back"]:
            rows = 4 if case["residual"] else 3   # dout, h, dx (dsum)
            return {"bytes": 2 * rows * n + 4 * T + weight + 4 * H, "flops": 10 * n}
        size = 6 if case["residual"] else 2       # x (residual, sum)
        size += {"bf16": 2, "fp8": 1 + 4 / 128, "both": 3 + 4 / 128}[case["out"]]
        return {"bytes": size * n + 4 * T + weight, "flops": (5 if case["out"] == "bf16" else 8) * n}
    if case["op"] == "route":
        E, k = case["experts"], case["k"]
        logit = 4 if case["logits"] == "fp32" else 2
        rows = T * E * logit * (2 if case["back"] else 1)
        return {"bytes": rows + T * k * 12 + (4 * E if case["bias"] else 0), "flops": 6 * T * E}
    H, E, k, I, G = (case[n] for n in ("hidden", "experts", "k", "inter", "group"))
    keep = 1 - case["drop"]
    read = E * (1 - (1 - k * keep / E) ** T)      # experts that are picked at least once, expected
    return {"bytes": read * 3 * H * I * (0.5 + 2 / G) + 4 * T * H + 12 * T * k, "flops": 6 * T * k * keep * H * I}


# ---- the definition in 64 bits ---------------------------------------------------------------


def exact(case, seed):
    i = inputs(case, seed)
    i = {n: v.double() if v is not None and v.is_floating_point() else v for n, v in i.items()}
    if case["op"] == "norm":
        return exact_norm(case, i)
    if case["op"] == "route":
        return exact_route(case, i)
    return exact_w4(case, i)


def exact_norm(c, i):
    H = c["hidden"]
    if c["back"]:
        # d(h_a rstd w_a)/d h_b = rstd w_a (a == b) - h_a w_a h_b rstd^3 / H
        up = i["dout"] * i["weight"]
        along = torch.einsum("th,th->t", up, i["h"]) * i["rstd"] ** 3 / H
        dx = torch.addcmul(up * i["rstd"][:, None], i["h"], along[:, None], value=-1)
        return {"dx": dx if i["dsum"] is None else dx + i["dsum"],
                "dweight": torch.einsum("th,th,t->h", i["dout"], i["h"], i["rstd"])}
    h = i["x"] if i["residual"] is None else i["x"] + i["residual"]
    ms = torch.einsum("th,th->t", h, h) / H
    y = h / torch.sqrt(ms + EPS)[:, None] * i["weight"]
    r = {"sum": None if i["residual"] is None else h, "rstd": (ms + EPS) ** -0.5}
    if c["out"] != "fp8":
        r["out"] = y
    if c["out"] != "bf16":
        blocks = y.unflatten(1, (H // 128, 128))
        top = torch.maximum(blocks.amax(2), -blocks.amin(2)).clamp(min=2.0 ** -100)
        r["scales"] = top / 448
        r["codes"] = (blocks / r["scales"][:, :, None]).flatten(1).float().to(torch.float8_e4m3fn)
    return r


def exact_route(c, i):
    E, k, n = c["experts"], c["k"], c["groups"]
    l = i["logits"]
    s = torch.sigmoid(l) if c["score"] == "sigmoid" else torch.softmax(l, 1).nan_to_num(0.0)
    if c["back"]:
        ids = i["ids"]
        picked = torch.zeros((len(l), E + 1), dtype=torch.bool, device=l.device)
        picked.scatter_(1, torch.where(ids < 0, E, ids), True)
        picked = picked[:, :E]
        g = torch.zeros((len(l), E + 1), dtype=l.dtype, device=l.device)
        g = g.scatter_(1, torch.where(ids < 0, E, ids), i["dweights"])[:, :E] * c["scale"] * picked
        if c["renorm"] and c["score"] == "softmax":   # a softmax over the picked logits alone
            q = torch.softmax(l.masked_fill(~picked, -math.inf), 1).nan_to_num(0.0)
            return q * (g - (q * g).sum(1, keepdim=True))
        if c["score"] == "softmax":
            return s * g - s * (s * g).sum(1, keepdim=True)
        if c["renorm"]:
            z = (s * picked).sum(1, keepdim=True)
            g = torch.where(z > 0, g / z - (s * g).sum(1, keepdim=True) / (z * z), torch.zeros_like(g)) * picked
        return g * s * torch.sigmoid(-l)
    key = l if not by_score(c) else torch.where(l == -math.inf, l, s if i["bias"] is None else s + i["bias"])
    order = torch.arange(E, device=l.device)
    if n > 1:
        two = key.unflatten(1, (n, E // n)).topk(min(2, E // n), 2)[0]
        by = two[:, :, 0] + (two[:, :, 1].clamp(min=-1e300) * (two[:, :, 1] > -1e300) if c["pair"] and E // n > 1 else 0)
        rank = (by[:, None, :] > by[:, :, None]).sum(2)
        same = (by[:, None, :] == by[:, :, None]) & (order[:n] < order[:n, None])
        out = (rank + same.sum(2)) >= c["kept"]
        key = torch.where(out.repeat_interleave(E // n, 1), -math.inf, key)
    ids = torch.full((len(l), k), -1, dtype=torch.int64, device=l.device)
    w = torch.zeros((len(l), k), dtype=l.dtype, device=l.device)
    for j in range(k):   # the largest, lowest index first, then without it
        best = key.amax(1, keepdim=True)
        at = torch.where(key == best, order, E).amin(1, keepdim=True)
        there = best > -math.inf
        ids[:, j:j + 1] = torch.where(there, at, -1)
        w[:, j:j + 1] = s.gather(1, at) * there
        key = key.scatter(1, at, -math.inf)
    if c["renorm"]:
        z = w.sum(1, keepdim=True)
        w = torch.where(z > 0, w / z, torch.zeros_like(w))
    return {"ids": ids, "weights": w * c["scale"]}


def exact_w4(c, i):
    I, G = c["inter"], c["group"]

    def matrix(codes, scales):
        m = torch.empty(codes.shape[0], codes.shape[1] * 2, dtype=torch.float64, device=codes.device)
        m[:, 0::2] = codes.remainder(16).double() - 8
        m[:, 1::2] = codes.div(16, rounding_mode="floor").double() - 8
        return m.unflatten(1, (-1, G)).mul_(scales[:, :, None]).flatten(1)

    out = torch.zeros(i["x"].shape, dtype=torch.float64, device=i["x"].device)
    for e in sorted(set(i["ids"].flatten().tolist()) - {-1}):
        t, j = (i["ids"] == e).nonzero(as_tuple=True)
        h = i["x"][t] @ matrix(i["w1"][e], i["s1"][e]).T
        a = h[:, :I] * torch.sigmoid(h[:, :I]) * h[:, I:]
        out.index_add_(0, t, i["weights"][t, j][:, None] * (a @ matrix(i["w2"][e], i["s2"][e]).T))
    return out
