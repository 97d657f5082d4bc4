"""A MoE block whose experts are computed on rows in expert order, with FP8 products:

    h, y    = residual + x, norm(h)                     moe_add_rmsnorm (bf16 and e4m3 rows)
    ids, w  = top-k of y gate^T                         moe_route_topk
    rows    = the e4m3 rows in expert order             moe_sort_picks, moe_sort_rows
    act     = silu(rows W1g^T) * (rows W1u^T), e4m3     moe_product_fp8, moe_swiglu_fp8
    experts = act W2^T                                  moe_product_fp8
    out     = sum of w * experts, and the shared expert moe_unsort_rows, moe_product_fp8

and, for training the router, the gradient of the routing weights and of the logits.
Run on a GB300:  python examples/grouped_experts.py [workload of gen.CONFIGS]
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import combine_topk_ids_gb300 as moe  # noqa: E402

EPS = 1e-6
BF, F8 = torch.bfloat16, torch.float8_e4m3fn


def empty(*shape, dtype=torch.float32):
    return torch.empty(shape, dtype=dtype, device="cuda")


def quantized(w):
    """e4m3 codes and block scales of bf16 weights [.., rows, cols]."""
    codes, scales = empty(*w.shape, dtype=F8), empty(*w.shape[:-2], -(-w.shape[-2] // 128), w.shape[-1] // 128)
    moe.moe_quantize_fp8(w, codes, scales, block_rows=128)
    return codes, scales


class Ffn:
    """silu(x Wg^T) * (x Wu^T) W2^T on e4m3 rows, for one expert (w1 [2I, H], w2 [H, I]) or for rows
    in expert order (w1 [E, 2I, H], w2 [E, H, I], with offsets).  Buffers for `rows` rows."""

    def __init__(self, rows, w1, w2):
        H, I = w2.shape[-2:]
        self.w1, self.w2 = quantized(w1), quantized(w2)
        self.gate_up, self.act, self.out = empty(rows, 2 * I, dtype=BF), empty(rows, I, dtype=F8), empty(rows, H, dtype=BF)
        self.scales = empty(rows, I // 128)

    def forward(self, codes, scales, status, offsets=None):
        live = None if offsets is None else offsets[-1:]
        moe.moe_product_fp8(codes, scales, *self.w1, self.gate_up, offsets=offsets, status=status)
        moe.moe_swiglu_fp8(self.gate_up, self.act, self.scales, live_rows=live)
        moe.moe_product_fp8(self.act, self.scales, *self.w2, self.out, offsets=offsets, status=status)
        return self.out


class GroupedBlock:
    """norm [H], gate [E, H], the experts' w1 and w2 and the shared expert's (bf16); router:
    moe.make_router(...).  Buffers for `tokens` rows."""

    def __init__(self, tokens, norm, gate, w1, w2, shared_w1, shared_w2, router):
        T, H, E, k = tokens, norm.shape[0], gate.shape[0], router.top_k
        self.norm, self.gate, self.router, self.E = norm, gate, router, E
        self.experts, self.shared = Ffn(T * k, w1, w2), Ffn(T, shared_w1, shared_w2)
        self.y, self.codes, self.scales = empty(T, H, dtype=BF), empty(T, H, dtype=F8), empty(T, H // 128)
        self.ids, self.weights = empty(T, k, dtype=torch.int64), empty(T, k)
        self.offsets, self.position = empty(E + 1, dtype=torch.int32), empty(T, k, dtype=torch.int32)
        self.workspace = empty(moe.moe_sort_picks_workspace_size(T, k, E), dtype=torch.uint8)
        self.rows, self.rows_scales = empty(T * k, H, dtype=F8), empty(T * k, H // 128)
        self.routed = empty(T, H, dtype=BF)
        self.status = empty(1, dtype=torch.int32)

    def forward(self, x, residual):
        """residual += x; the block's output, which is valid if check() finds nothing.  The order of the picks
        writes the status word, and the products after it add to it."""
        moe.moe_add_rmsnorm(x, residual, self.norm, EPS, sum_out=residual, out=self.y, out_fp8=self.codes,
                            scales=self.scales)
        self.logits = torch.mm(self.y, self.gate.t()).float()
        moe.moe_route_topk(self.router, self.logits, None, self.ids, self.weights)
        moe.moe_sort_picks(self.ids, self.E, self.offsets, self.position, self.workspace, status=self.status)
        moe.moe_sort_rows(self.codes, self.position, self.rows, x_scales=self.scales, rows_scales=self.rows_scales)
        self.experts.forward(self.rows, self.rows_scales, self.status, self.offsets)
        moe.moe_unsort_rows(self.experts.out, self.weights, self.position, self.routed)
        return self.routed + self.shared.forward(self.codes, self.scales, self.status)

    def check(self):
        """Raises where the last forward met a bad expert id or a product's wait gave up (synchronises)."""
        bits = self.status.item()
        if bits:
            raise RuntimeError("the forward is invalid: status 0x%x (moe.STATUS_*)" % bits)

    def router_backward(self, dout):
        """d(routing weights) and d(logits) of the last forward, from the output's gradient."""
        dweights, dlogits = torch.empty_like(self.weights), torch.empty_like(self.logits)
        moe.moe_unsort_rows_backward(dout, self.experts.out, self.weights, self.position, None, dweights)
        moe.moe_route_topk_backward(self.router, self.logits, self.ids, dweights, dlogits)
        return dweights, dlogits


def make(cfg, tokens, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape, scale=1.0):
        return torch.randn(shape, generator=g, device="cuda", dtype=BF) * scale

    E, H, I = cfg.E, cfg.H, cfg.I
    block = GroupedBlock(tokens, randn(H, scale=0.1) + 1, randn(E, H, scale=H ** -0.5),
                         randn(E, 2 * I, H, scale=H ** -0.5), randn(E, H, I, scale=I ** -0.5),
                         randn(2 * I, H, scale=H ** -0.5), randn(H, I, scale=I ** -0.5),
                         moe.make_router(E, cfg.k, "sigmoid", scale=2.5))
    return block, randn(tokens, H), randn(tokens, H)


def main():
    import gen
    cfg = gen.CONFIGS[sys.argv[1] if len(sys.argv) > 1 else "tiny_ll_em"]
    for tokens in (1, cfg.tokens):
        block, x, residual = make(cfg, tokens)
        out = block.forward(x, residual)
        block.check()
        dweights, dlogits = block.router_backward(torch.ones_like(out))
        print("%d tokens: |out| %.4f, |dweights| %.4f, |dlogits| %.4f"
              % (tokens, out.float().norm(), dweights.norm(), dlogits.norm()))


if __name__ == "__main__":
    main()
