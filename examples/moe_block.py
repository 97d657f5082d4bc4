"""One MoE block of a decoder, from the residual stream to the residual stream:

    h, y   = residual + x, norm(h)            moe_add_rmsnorm
    logits = y gate^T                         torch
    ids, w = top-k of the logits              moe_route_topk
    x'     = sum of the picked experts        MoELayerW4 (decode)  or
                                              dispatch_fp8 -> expert_ffn -> combine (prefill)

and, for training the parts around the experts, the gradients of the routing weights and of the
norm.  Run on a GB300:  python examples/moe_block.py [workload of gen.CONFIGS] [tokens to decode]
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import combine_topk_ids_gb300 as moe  # noqa: E402

EPS = 1e-6


class MoEBlock:
    """Weights of one block and the buffers for `tokens` rows.  norm: [H], gate: [E, H] (bf16);
    bias: float32 [E] (load balance) or None; router: moe.make_router(...)."""

    def __init__(self, tokens, norm, gate, bias, router):
        T, H, dev = tokens, norm.shape[0], norm.device
        self.norm, self.gate, self.bias, self.router = norm, gate, bias, router
        self.y = torch.empty((T, H), dtype=torch.bfloat16, device=dev)
        self.codes = torch.empty((T, H), dtype=torch.float8_e4m3fn, device=dev)
        self.scales = torch.empty((T, H // 128), device=dev)
        self.rstd = torch.empty(T, device=dev)
        self.ids = torch.empty((T, router.top_k), dtype=torch.int64, device=dev)
        self.weights = torch.empty((T, router.top_k), device=dev)

    def _route(self):
        self.logits = torch.mm(self.y, self.gate.t()).float()
        moe.moe_route_topk(self.router, self.logits, self.bias, self.ids, self.weights)

    def decode(self, x, residual, layer):
        """residual += x; the block's output from `layer` (MoELayerW4)."""
        moe.moe_add_rmsnorm(x, residual, self.norm, EPS, sum_out=residual, out=self.y)
        self._route()
        return layer.forward(self.y, self.ids, self.weights)

    def prefill(self, x, residual, layer):
        """The same from `layer` (MoELayer1GPU, quant="fp8"): the norm's e4m3 rows go to the
        experts as they are, its bf16 rows to the gate."""
        moe.moe_add_rmsnorm(x, residual, self.norm, EPS, sum_out=residual, out=self.y, out_fp8=self.codes,
                            scales=self.scales, rstd=self.rstd)
        self._route()
        layer.dispatch_fp8(self.codes, self.scales, self.ids, self.weights)
        layer.expert_ffn()
        return layer.combine(self.weights)

    def backward(self, h, dweights, dy, dresidual):
        """Gradients behind the routing weights and the norm after prefill: dweights of
        self.weights, dy of the rows that went to the experts, dresidual of the residual stream
        h (what prefill left there).  Returns d(x and residual), d(norm), d(gate)."""
        dlogits = torch.empty_like(self.logits)
        moe.moe_route_topk_backward(self.router, self.logits, self.ids, dweights, dlogits)
        dlogits = dlogits.bfloat16()
        dgate = torch.mm(dlogits.t(), self.y)
        dout = torch.addmm(dy, dlogits, self.gate)
        dx, dnorm = torch.empty_like(h), torch.empty(h.shape[1], device=h.device)
        work = torch.empty(moe.moe_add_rmsnorm_workspace_size(*h.shape), dtype=torch.uint8, device=h.device)
        moe.moe_add_rmsnorm_backward(dout, h, self.norm, self.rstd, dx, dnorm, work, dsum=dresidual)
        return dx, dnorm, dgate


def main():
    import gen
    cfg = gen.CONFIGS[sys.argv[1] if len(sys.argv) > 1 else "tiny_ll_em"]
    tokens = int(sys.argv[2]) if len(sys.argv) > 2 else 4
    g = torch.Generator(device="cuda").manual_seed(0)

    def randn(*shape, scale=1.0):
        return (torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16) * scale)

    norm, gate = randn(cfg.H, scale=0.1) + 1, randn(cfg.E, cfg.H, scale=cfg.H ** -0.5)
    w1, w2 = randn(cfg.E, 2 * cfg.I, cfg.H, scale=cfg.H ** -0.5), randn(cfg.E, cfg.H, cfg.I, scale=cfg.I ** -0.5)
    bias = torch.zeros(cfg.E, device="cuda")
    router = moe.make_router(cfg.E, cfg.k, "sigmoid", scale=1.0)

    experts = moe.MoELayerW4(tokens, cfg.H, cfg.E, cfg.k, cfg.I, group=128)
    experts.quantize_weights(w1, w2)
    block = MoEBlock(tokens, norm, gate, bias, router)
    x, residual = randn(tokens, cfg.H), randn(tokens, cfg.H)
    out = block.decode(x, residual, experts)
    print("decode: %d tokens, status %d, |out| %.4f" % (tokens, experts.status(), out.float().norm()))

    layer = moe.MoELayer1GPU(cfg.W, cfg.Tr, cfg.tokens, cfg.H, cfg.E, cfg.k, cfg.I, cfg.layout, cfg.algo, quant="fp8")
    layer.set_weights(w1, w2)
    block = MoEBlock(cfg.tokens, norm, gate, bias, router)
    x, residual = randn(cfg.tokens, cfg.H), randn(cfg.tokens, cfg.H)
    out = block.prefill(x, residual, layer)
    print("prefill: %d tokens, status %d, |out| %.4f" % (cfg.tokens, layer.status(), out.float().norm()))
    dx, dnorm, dgate = block.backward(residual, torch.rand_like(block.weights), out, torch.zeros_like(residual))
    print("backward: |dx| %.4f, |dnorm| %.4f, |dgate| %.4f" % (dx.float().norm(), dnorm.norm(), dgate.float().norm()))


if __name__ == "__main__":
    main()
