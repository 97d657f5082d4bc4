"""The measured cases of the operators on expert-grouped rows.

sort      a batch's picks in expert order and their rows gathered into it (bf16, float32, or
          e4m3 codes with a scale per 128 columns), and the rows' gradient
unsort    the rows back in token order, weighted and summed over a token's picks, and the
          gradient in the rows and in the weights
product   e4m3 rows times e4m3 weights with a scale per 128 columns and per 128 x 128 block,
          one weight matrix or one for each expert's rows
quantize  rows or weights to e4m3 codes and scales, and SwiGLU with such an output

With `own` false, run() computes the plain form with elementary torch operations in 32
bits; with `own` true it calls combine_topk_ids_gb300.
"""
import math

import torch

own = False

TYPE = {"bf16": torch.bfloat16, "fp32": torch.float32, "fp8": torch.float8_e4m3fn}
SIZE = {"bf16": 2, "fp32": 4, "fp8": 1 + 4 / 128}


def listed():
    return [
        # the decode batch of the 256-expert model on its way to the experts: all latency
        sort("sort_decode", 64, 7168, 256, 8),
        # the prefill batch (8 x 4096 tokens), the codes and scales that the norm has written
        sort("sort_prefill_fp8", 32768, 7168, 256, 8, dtype="fp8"),
        # the decode batch's expert outputs back to its tokens
        unsort("unsort_decode", 64, 7168, 256, 8),
        # the same for the prefill batch
        unsort("unsort_prefill", 32768, 7168, 256, 8),
        # a training step of the ragged workload's layer: rows one column short of it, so that
        # hardly any starts on a 16-byte boundary, one pick in ten masked
        unsort("unsort_backward", 16381, 2047, 128, 4, drop=0.1, back=True),
        # one token through the shared expert's gate and up projection of the 256-expert model
        product("product_one_token", 1, 4096, 7168),
        # the prefill batch through it
        product("product_prefill", 32768, 4096, 7168),
        # the decode batch's 512 picks through the 256 experts' gate and up projections: about
        # two rows for each, all weights read
        product("product_experts_decode", 64, 4096, 7168, experts=256, k=8),
        # a prompt of 8192 tokens through the experts' down projections, 256 rows for each
        product("product_experts_prefill", 8192, 7168, 2048, experts=256, k=8),
        # a ragged batch and an output width that no tile divides
        product("product_ragged", 777, 1003, 1408, out="fp32"),
        # the activation between the shared expert's two products, over the prefill batch
        quantize("swiglu_prefill", 32768, 2048, swiglu=True),
        # a decode batch's bf16 rows in front of a product
        quantize("quantize_decode", 64, 7168),
    ]


def sort(name, tokens, hidden, experts, k, dtype="bf16", drop=0.0, back=False):
    return {"name": name, "op": "sort", "back": back, "tokens": tokens, "hidden": hidden, "experts": experts,
            "k": k, "dtype": dtype, "drop": drop}


def unsort(name, tokens, hidden, experts, k, dtype="bf16", out="bf16", drop=0.0, back=False):
    return {"name": name, "op": "unsort", "back": back, "tokens": tokens, "hidden": hidden, "experts": experts,
            "k": k, "dtype": dtype, "out": out, "drop": drop}


def product(name, tokens, n, inner, experts=0, k=1, out="bf16", drop=0.0):
    return {"name": name, "op": "product", "tokens": tokens, "n": n, "inner": inner, "experts": experts, "k": k,
            "out": out, "drop": drop}


def quantize(name, rows, cols, dtype="bf16", block=1, swiglu=False):
    return {"name": name, "op": "quantize", "rows": rows, "cols": cols, "dtype": dtype, "block": block,
            "swiglu": swiglu}


def draw(rng):
    def spread(lo, hi):   # even over the logarithm
        return round(math.exp(rng.uniform(math.log(lo), math.log(hi))))

    def of128(lo, hi):
        return 128 * max(1, round(spread(lo, hi) / 128))

    op = rng.choice(("sort", "unsort", "product", "product", "quantize"))
    drop = rng.choice((0.0, 0.0, 0.1, 0.5))
    experts = rng.choice((4, 8, 16, 32, 60, 64, 128, 160, 256, 384))
    k = rng.randint(1, min(8, experts))
    while True:
        if op == "sort":
            dtype, back = rng.choice(("bf16", "fp8", "fp32")), rng.random() < 0.3
            dtype = "bf16" if back and dtype == "fp8" else dtype
            hidden = of128(128, 8192) if dtype == "fp8" or rng.random() < 0.6 else spread(32, 8192)
            case = sort("", spread(1, 32768), hidden, experts, k, dtype, drop, back)
            fits = case["tokens"] * k * hidden * SIZE[dtype] <= 32768 * 8 * 7168
        elif op == "unsort":
            hidden = of128(128, 8192) if rng.random() < 0.6 else spread(32, 8192)
            case = unsort("", spread(1, 32768), hidden, experts, k, rng.choice(("bf16", "fp32")),
                          rng.choice(("bf16", "bf16", "fp32")), drop, rng.random() < 0.4)
            fits = case["tokens"] * k * hidden * SIZE[case["dtype"]] <= 32768 * 8 * 7168
        elif op == "product":
            many = rng.random() < 0.5
            n = of128(128, 8192) if rng.random() < 0.7 else spread(8, 8192)
            case = product("", spread(1, 32768), n, of128(128, 14336), experts if many else 0, k if many else 1,
                           rng.choice(("bf16", "bf16", "fp32")), drop if many else 0.0)
            fits = (case["tokens"] * case["k"] * n * case["inner"] <= 32768 * 4096 * 7168
                    and max(1, case["experts"]) * n * case["inner"] <= 256 * 4096 * 7168
                    and case["tokens"] * case["k"] * (case["inner"] + 4 * n) <= 32768 * 8 * 7168)
        else:
            swiglu = rng.random() < 0.5
            case = quantize("", spread(1, 32768), of128(128, 14336), rng.choice(("bf16", "fp32")),
                            1 if swiglu else rng.choice((1, 1, 128)), swiglu)
            fits = case["rows"] * case["cols"] <= 32768 * 7168
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
    return {"sort": sort_inputs, "unsort": unsort_inputs, "product": product_inputs,
            "quantize": quantize_inputs}[case["op"]](case, generator(seed))


def rows_like(shape, g, dtype=torch.bfloat16):
    """Rows of different size, as a layer's tokens have them."""
    v = torch.randn(shape, generator=g, device="cuda", dtype=dtype)
    return v.mul_(torch.rand((shape[0], 1), generator=g, device="cuda").mul_(2).exp_().to(dtype))


def picks(c, g):
    """int64 ids [T, k], -1 where masked: experts are not equally liked, no token has one twice."""
    T, E, k = c["tokens"], c["experts"], c["k"]
    like = torch.rand(E, generator=g, device="cuda").mul_(2).exp_()
    # the k smallest of exponential variables: k experts without repetition, in proportion to `like`
    clock = torch.rand((T, E), generator=g, device="cuda").clamp_(min=1e-30).log_().neg_().div_(like)
    ids = clock.argsort(1)[:, :k].contiguous()
    if c["drop"]:
        ids[torch.rand((T, k), generator=g, device="cuda") < c["drop"]] = -1
    return ids


def order_of(ids, experts):
    """offsets [E + 1], position [T, k] and source [T k] of the picks in (expert, token, pick) order."""
    flat = torch.where(ids < 0, experts, ids).flatten()
    order = flat.sort(stable=True)[1]
    n = torch.arange(len(flat), device=ids.device)
    position = torch.empty_like(flat).scatter_(0, order, n).view(ids.shape).masked_fill_(ids < 0, -1)
    offsets = (flat[None, :] < torch.arange(experts + 1, device=ids.device)[:, None]).sum(1)
    return offsets.int(), position.int(), order.masked_fill(n >= offsets[-1], -1).int()


def codes_of(v, g, block):
    """e4m3 codes and scales of a matrix [.., rows, cols]; block: rows that share a scale."""
    rows, cols = v.shape[-2:]
    full = torch.nn.functional.pad(v, (0, 0, 0, -rows % block)).unflatten(-1, (-1, 128)).unflatten(-3, (-1, block))
    scale = full.abs().float().amax((-3, -1)).clamp_(min=2.0 ** -100).div_(448)
    full = full.float().div_(scale[..., :, None, :, None]).to(torch.float8_e4m3fn)
    return full.flatten(-4, -3).flatten(-2)[..., :rows, :].contiguous(), scale


def sort_inputs(c, g):
    T, H, P = c["tokens"], c["hidden"], c["tokens"] * c["k"]
    ids = picks(c, g)
    if c["back"]:
        return {"position": order_of(ids, c["experts"])[1], "drows": rows_like((P, H), g, TYPE[c["dtype"]])}
    if c["dtype"] == "fp8":
        x, scales = codes_of(rows_like((T, H), g), g, 1)
        return {"ids": ids, "x": x, "x_scales": scales}
    return {"ids": ids, "x": rows_like((T, H), g, TYPE[c["dtype"]]), "x_scales": None}


def unsort_inputs(c, g):
    T, H, k = c["tokens"], c["hidden"], c["k"]
    w = torch.rand((T, k), generator=g, device="cuda").add_(0.05)
    i = {"position": order_of(picks(c, g), c["experts"])[1], "weights": w.div_(w.sum(1, keepdim=True)),
         "rows": rows_like((T * k, H), g, TYPE[c["dtype"]])}
    if c["back"]:
        i["dout"] = torch.randn((T, H), generator=g, device="cuda").mul_(0.01).to(TYPE[c["out"]])
    return i


def product_inputs(c, g):
    M, N, K, E = c["tokens"] * c["k"], c["n"], c["inner"], c["experts"]
    i = {"offsets": None, "counts": None}
    if E:
        i["offsets"] = order_of(picks(c, g), E)[0]
        i["counts"] = i["offsets"].diff().tolist()   # for the plain form, which takes expert by expert
    i["a"], i["a_scales"] = codes_of(rows_like((M, K), g), g, 1)

    def weights():
        return codes_of(torch.randn((N, K), generator=g, device="cuda", dtype=torch.bfloat16).mul_(K ** -0.5), g, 128)

    if E:
        i["b"] = torch.empty((E, N, K), dtype=torch.float8_e4m3fn, device="cuda")
        i["b_scales"] = torch.empty((E, -(-N // 128), K // 128), device="cuda")
        for e in range(E):
            i["b"][e], i["b_scales"][e] = weights()
    else:
        i["b"], i["b_scales"] = weights()
    return i


def quantize_inputs(c, g):
    rows, cols = c["rows"], c["cols"] * (2 if c["swiglu"] else 1)
    return {"x": rows_like((rows, cols), g, TYPE[c["dtype"]])}


def prepare(case, seed):
    s = {"case": case, **inputs(case, seed)}
    if not own:
        return s
    import combine_topk_ids_gb300 as moe

    s["moe"] = moe

    def empty(*shape, dtype=torch.float32):
        return torch.empty(shape, dtype=dtype, device="cuda")

    def zeros(*shape, dtype=torch.float32):   # rows that belong to no pick stay as they are
        return torch.zeros(shape, dtype=dtype, device="cuda")

    c = case
    if c["op"] in ("sort", "unsort"):
        T, H, k, E = c["tokens"], c["hidden"], c["k"], c["experts"]
    if c["op"] == "sort":
        if c["back"]:
            s["dx"] = empty(T, H, dtype=TYPE[c["dtype"]])
            return s
        s["offsets"], s["position"] = empty(E + 1, dtype=torch.int32), empty(T, k, dtype=torch.int32)
        s["source"] = empty(T * k, dtype=torch.int32)
        s["workspace"] = empty(moe.moe_sort_picks_workspace_size(T, k, E), dtype=torch.uint8)
        s["rows"] = zeros(T * k, H, dtype=torch.uint8 if c["dtype"] == "fp8" else TYPE[c["dtype"]])
        if c["dtype"] == "fp8":
            s["rows"] = s["rows"].view(torch.float8_e4m3fn)
        s["rows_scales"] = zeros(T * k, H // 128) if c["dtype"] == "fp8" else None
    elif c["op"] == "unsort":
        if c["back"]:
            s["drows"], s["dweights"] = zeros(T * k, H, dtype=TYPE[c["dtype"]]), empty(T, k)
        else:
            s["out"] = empty(T, H, dtype=TYPE[c["out"]])
    elif c["op"] == "product":
        s["out"] = zeros(len(s["a"]), c["n"], dtype=TYPE[c["out"]])
    else:
        s["codes"] = empty(c["rows"], c["cols"], dtype=torch.float8_e4m3fn)
        s["scales"] = empty(-(-c["rows"] // c["block"]), c["cols"] // 128)
    return s


# ---- one pass --------------------------------------------------------------------------------


def run(s):
    c = s["case"]
    if c["op"] == "sort":
        return (sort_back if c["back"] else sort_run)(s)
    if c["op"] == "unsort":
        return (unsort_back if c["back"] else unsort_run)(s)
    return product_run(s) if c["op"] == "product" else quantize_run(s)


def sort_run(s):
    c = s["case"]
    if own:
        s["moe"].moe_sort_picks(s["ids"], c["experts"], s["offsets"], s["position"], s["workspace"], source=s["source"])
        s["moe"].moe_sort_rows(s["x"], s["position"], s["rows"], x_scales=s["x_scales"], rows_scales=s["rows_scales"])
        return {n: s[n] for n in ("offsets", "position", "source", "rows", "rows_scales")}
    offsets, position, source = order_of(s["ids"], c["experts"])

    def gather(x):
        if x is None:
            return None
        x = x.view(torch.uint8) if x.dtype == torch.float8_e4m3fn else x
        return x[source.clamp_min(0) // c["k"]].masked_fill_(source[:, None] < 0, 0)

    rows = gather(s["x"])
    return {"offsets": offsets, "position": position, "source": source, "rows": rows.view(s["x"].dtype),
            "rows_scales": gather(s["x_scales"])}


def sort_back(s):
    if own:
        s["moe"].moe_sort_rows_backward(s["drows"], s["position"], s["dx"])
        return s["dx"]
    return gathered_sum(s["drows"], None, s["position"]).to(s["drows"].dtype)


def gathered_sum(rows, weights, position):
    out = torch.zeros((len(position), rows.shape[1]), device=rows.device)
    for j in range(position.shape[1]):
        p = position[:, j]
        r = rows[p.clamp_min(0)].float()
        if weights is not None:
            r = r * weights[:, j, None]
        out += r.masked_fill_(p[:, None] < 0, 0)
    return out


def unsort_run(s):
    if own:
        s["moe"].moe_unsort_rows(s["rows"], s["weights"], s["position"], s["out"])
        return s["out"]
    return gathered_sum(s["rows"], s["weights"], s["position"]).to(TYPE[s["case"]["out"]])


def unsort_back(s):
    if own:
        s["moe"].moe_unsort_rows_backward(s["dout"], s["rows"], s["weights"], s["position"], s["drows"], s["dweights"])
        return {"drows": s["drows"], "dweights": s["dweights"]}
    dout, position = s["dout"].float(), s["position"]
    drows, dweights = torch.zeros_like(s["rows"]), torch.zeros_like(s["weights"])
    for j in range(position.shape[1]):
        t = (position[:, j] >= 0).nonzero()[:, 0]
        p = position[t, j]
        dweights[t, j] = (dout[t] * s["rows"][p]).sum(1)
        drows[p] = (dout[t] * s["weights"][t, j, None]).to(drows.dtype)
    return {"drows": drows, "dweights": dweights}


def matrix(codes, scales, block):
    """The matrix that codes and scales stand for, in 32 bits."""
    return codes.float() * scales.repeat_interleave(block, 0)[:len(codes)].repeat_interleave(128, 1)


def product_run(s):
    if own:
        s["moe"].moe_product_fp8(s["a"], s["a_scales"], s["b"], s["b_scales"], s["out"], offsets=s["offsets"])
        return s["out"]
    dtype = TYPE[s["case"]["out"]]
    a = matrix(s["a"], s["a_scales"], 1)
    if s["offsets"] is None:
        return (a @ matrix(s["b"], s["b_scales"], 128).T).to(dtype)
    out = torch.zeros((len(a), s["case"]["n"]), dtype=dtype, device=a.device)
    begin = 0
    for e, n in enumerate(s["counts"]):
        if n:
            out[begin:begin + n] = a[begin:begin + n] @ matrix(s["b"][e], s["b_scales"][e], 128).T
        begin += n
    return out


def quantize_run(s):
    c = s["case"]
    if own:
        if c["swiglu"]:
            s["moe"].moe_swiglu_fp8(s["x"], s["codes"], s["scales"])
        else:
            s["moe"].moe_quantize_fp8(s["x"], s["codes"], s["scales"], block_rows=c["block"])
        return {"codes": s["codes"], "scales": s["scales"]}
    v = s["x"].float()
    if c["swiglu"]:
        gate, up = v.split(c["cols"], 1)
        v = gate / (1 + torch.exp(-gate)) * up
    v = torch.nn.functional.pad(v, (0, 0, 0, -c["rows"] % c["block"])).view(-1, c["block"], c["cols"] // 128, 128)
    a = v.abs().amax((1, 3)).clamp_min(2.0 ** -100)
    codes = (v * (448 / a)[:, None, :, None]).to(torch.float8_e4m3fn)
    return {"codes": codes.view(-1, c["cols"])[:c["rows"]], "scales": a / 448}


# ---- what a pass cannot do without -----------------------------------------------------------


def work(case):
    c = case
    if c["op"] in ("sort", "unsort"):
        T, P = c["tokens"], c["tokens"] * c["k"]
        n = T * c["hidden"]
        there = P * (1 - c["drop"]) * c["hidden"]   # elements of the rows that picks have, expected
        size = SIZE[c["dtype"]]
        if c["op"] == "sort":
            plan = 4 * P if c["back"] else 16 * P + 4 * c["experts"]   # position, or ids, position and source
            return {"bytes": size * (n + there) + plan, "flops": there if c["back"] else 0}
        if c["back"]:
            return {"bytes": SIZE[c["out"]] * n + 2 * size * there + 12 * P, "flops": 3 * there}
        return {"bytes": SIZE[c["out"]] * n + size * there + 8 * P, "flops": 2 * there}
    if c["op"] == "product":
        N, K, E = c["n"], c["inner"], c["experts"]
        M = c["tokens"] * c["k"] * (1 - c["drop"])
        read = 1
        if E:   # experts with a row at all, were they equally liked
            read = E * (1 - (1 - c["k"] * (1 - c["drop"]) / E) ** c["tokens"])
        bytes_ = M * K * SIZE["fp8"] + read * N * K * (1 + 4 / 128 ** 2) + M * N * SIZE[c["out"]]
        return {"bytes": bytes_, "flops": 2 * M * N * K}
    n = c["rows"] * c["cols"]
    size = SIZE[c["dtype"]] * (2 if c["swiglu"] else 1)
    return {"bytes": n * (size + 1 + 4 / 128 / c["block"]), "flops": n * (8 if c["swiglu"] else 3)}


# ---- the definition in 64 bits ---------------------------------------------------------------


def exact(case, seed):
    i = inputs(case, seed)
    return {"sort": exact_sort, "unsort": exact_unsort, "product": exact_product,
            "quantize": exact_quantize}[case["op"]](case, i)


def exact_order(ids, E):
    """Picks by counting: a pick comes after those of smaller experts and the earlier ones of its own."""
    offsets, position = [0], torch.full_like(ids, -1).flatten()
    flat = ids.flatten()
    source = torch.full_like(flat, -1)
    for e in range(E):
        own_picks = (flat == e).nonzero().flatten()
        at = offsets[-1] + torch.arange(len(own_picks), device=ids.device)
        position[own_picks], source[at] = at, own_picks
        offsets.append(offsets[-1] + len(own_picks))
    return torch.tensor(offsets, dtype=torch.int32, device=ids.device), position.view(ids.shape).int(), source.int()


def exact_sort(c, i):
    if c["back"]:
        return summed(i["drows"], None, i["position"])
    offsets, position, source = exact_order(i["ids"], c["experts"])
    there = int(offsets[-1])
    token = source[:there].long() // c["k"]

    def gather(x):
        if x is None:
            return None
        x = x.double() if x.dtype != torch.float8_e4m3fn else x.float()
        out = torch.zeros((len(source), x.shape[1]), dtype=x.dtype, device=x.device)
        out[:there] = x.index_select(0, token)
        return out

    rows = gather(i["x"])
    return {"offsets": offsets, "position": position, "source": source,
            "rows": rows.to(i["x"].dtype) if c["dtype"] == "fp8" else rows, "rows_scales": gather(i["x_scales"])}


def summed(rows, weights, position):
    T, k = position.shape
    t, j = (position >= 0).nonzero(as_tuple=True)
    out = torch.zeros((T, rows.shape[1]), dtype=torch.float64, device=rows.device)
    for b in range(0, len(t), 16384):   # picks in pieces: rows in 64 bits are large
        tt, jj = t[b:b + 16384], j[b:b + 16384]
        r = rows[position[tt, jj].long()].double()
        out.index_add_(0, tt, r if weights is None else r * weights[tt, jj].double()[:, None])
    return out


def exact_unsort(c, i):
    if not c["back"]:
        return summed(i["rows"], i["weights"], i["position"])
    t, j = (i["position"] >= 0).nonzero(as_tuple=True)
    at = i["position"][t, j].long()
    drows = torch.zeros(i["rows"].shape, dtype=torch.float64, device=at.device)
    dweights = torch.zeros(i["weights"].shape, dtype=torch.float64, device=at.device)
    for b in range(0, len(t), 16384):
        tt, jj, a = t[b:b + 16384], j[b:b + 16384], at[b:b + 16384]
        d = i["dout"][tt].double()
        drows[a] = torch.einsum("ph,p->ph", d, i["weights"][tt, jj].double())
        dweights[tt, jj] = torch.einsum("ph,ph->p", d, i["rows"][a].double())
    return {"drows": drows, "dweights": dweights}


def exact_product(c, i):
    out = torch.zeros((len(i["a"]), c["n"]), dtype=torch.float64, device=i["a"].device)
    counts = i["counts"] if i["offsets"] is not None else [len(i["a"])]
    weights = [(i["b"], i["b_scales"])] if i["offsets"] is None else zip(i["b"], i["b_scales"])
    begin = 0
    for n, (b, sb) in zip(counts, weights):
        there = slice(begin, begin + n)
        begin += n
        if not n:
            continue
        # block by block of the inner dimension: (codes times codes) times both scales
        for q in range(c["inner"] // 128):
            cols = slice(128 * q, 128 * q + 128)
            part = i["a"][there, cols].double() @ b[:, cols].double().T
            part *= i["a_scales"][there, q, None].double()
            out[there] += part * sb[:, q].double().repeat_interleave(128)[:c["n"]]
    return out


def exact_quantize(c, i):
    v = i["x"].double()
    if c["swiglu"]:
        v = v[:, :c["cols"]] * torch.sigmoid(v[:, :c["cols"]]) * v[:, c["cols"]:]
    codes = torch.empty(v.shape, dtype=torch.float8_e4m3fn, device=v.device)
    scales = torch.empty((-(-c["rows"] // c["block"]), c["cols"] // 128), dtype=torch.float64, device=v.device)
    for b in range(c["cols"] // 128):
        part = v[:, 128 * b:128 * b + 128]
        top = torch.maximum(part.amax(1), -part.amin(1))
        if c["block"] > 1:
            top = torch.stack([t.max() for t in top.split(c["block"])])
        scales[:, b] = top.clamp(min=2.0 ** -100) / 448
        per_row = scales[:, b].repeat_interleave(c["block"])[:c["rows"], None]
        codes[:, 128 * b:128 * b + 128] = (part / per_row).float().to(torch.float8_e4m3fn)
    return {"codes": codes, "scales": scales}
