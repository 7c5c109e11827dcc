"""One mixture-of-experts layer served and its router trained, with adapters of
several requests beside the shared projections, from this package's operators:

    python examples/moe_layer.py [--tokens T] [--requests N]

    o = FP8 projection of the attention output + each request's adapter   lora_linear
    routing of o's rows to k experts                                      moe_route
    shared expert: gate/up (with adapters), SwiGLU, down                  lora_linear, linear
    routed experts on the rows listed by expert, added to the shared one  moe_experts
    the router's gradient from the output's and from the balance loss     moe_combine_backward,
                                                                          moe_route_backward
Random weights; the sizes are small.
"""
import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import block_scaled_fp8_act_amd as fb  # noqa: E402

HIDDEN, INTER, EXPERTS, TOPK, ADAPTERS, RANK = 1024, 512, 32, 4, 8, 16


class Layer:
    """The layer's weights: FP8 blocks with their scales, a fp32 router, and
    the adapters of the two adapted projections."""

    def __init__(self, device="cuda", seed=0):
        g = torch.Generator(device=device).manual_seed(seed)
        rand = lambda *s: torch.randn(*s, device=device, generator=g)  # noqa: E731
        block = lambda n, k: fb.weight_block_quant((rand(n, k) * k ** -0.5).bfloat16())  # noqa: E731
        stack = lambda ws: tuple(torch.stack(t) for t in zip(*ws))  # noqa: E731
        self.o = block(HIDDEN, HIDDEN)
        self.shared_up, self.shared_down = block(2 * INTER, HIDDEN), block(HIDDEN, INTER)
        self.up = stack([block(2 * INTER, HIDDEN) for _ in range(EXPERTS)])
        self.down = stack([block(HIDDEN, INTER) for _ in range(EXPERTS)])
        self.router = rand(EXPERTS, HIDDEN) * HIDDEN ** -0.5
        low = lambda n: ((rand(ADAPTERS, RANK, HIDDEN) * HIDDEN ** -0.5).bfloat16(),  # noqa: E731
                         (rand(ADAPTERS, n, RANK) * 0.1).bfloat16())
        self.o_adapters, self.up_adapters = low(HIDDEN), low(2 * INTER)
        self.scale = torch.full((ADAPTERS,), 2.0, device=device)

    def forward(self, x, adapter, mask=None, loss_coef=None):
        """x [T, HIDDEN] bf16, adapter [T] int32 (-1: none) -> (y, routing, h)."""
        # larger batches list their rows by adapter once, for every projection
        groups = fb.group_rows(adapter, ADAPTERS) if len(x) > 64 else None
        h = fb.lora_linear(x, *self.o, *self.o_adapters, adapter, self.scale, groups)
        routing = fb.moe_route(h.float() @ self.router.t(), TOPK, mask=mask, loss_coef=loss_coef)
        up = fb.lora_linear(h, *self.shared_up, *self.up_adapters, adapter, self.scale, groups)
        shared = fb.block_gemm(*fb.swiglu_act_quant(up), *self.shared_down)
        return fb.moe_experts(h, routing, *self.up, *self.down, shared), routing, h

    def router_gradient(self, h, routing, d_y):
        """Gradient of the router's weights: through the experts' weighted sum
        and the balance loss (the FP8 products themselves are not trained)."""
        groups = fb.group_rows(routing.ids, EXPERTS)
        rows = h.index_select(0, groups.order // TOPK)
        hidden = fb.grouped_block_gemm(*fb.act_quant_group(rows), *self.up, groups.offsets)
        y = fb.grouped_block_gemm(*fb.swiglu_act_quant(hidden), *self.down, groups.offsets)
        _, d_weights = fb.moe_combine_backward(d_y, y, routing.weights, groups.positions,
                                               groups.offsets)
        logits = h.float() @ self.router.t()
        d_logits = fb.moe_route_backward(logits, routing, d_weights,
                                         torch.ones(1, device=h.device))
        return d_logits.t() @ h.float()


def main(argv=None):
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("--tokens", type=int, default=200)
    p.add_argument("--requests", type=int, default=12)
    a = p.parse_args(argv)
    layer = Layer()
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(a.tokens, HIDDEN, device="cuda", generator=g).bfloat16()
    request = torch.arange(a.tokens, device="cuda") * a.requests // a.tokens
    adapter = (request % (ADAPTERS + 1) - 1).int()          # every ninth request has none
    y, routing, h = layer.forward(x, adapter, loss_coef=0.01)
    print(f"served {a.tokens} tokens of {a.requests} requests: output {tuple(y.shape)}, "
          f"rows per expert {int(routing.counts.min())} to {int(routing.counts.max())}")
    one, _, _ = layer.forward(x[:1], adapter[:1])
    print(f"one token alone: largest difference {float((one - y[:1]).abs().max()):.4f}")
    before = float(routing.loss)
    d_router = layer.router_gradient(h, routing, torch.zeros_like(y))
    for _ in range(20):                                      # the balance loss alone
        layer.router -= 20.0 * d_router
        routing = fb.moe_route(h.float() @ layer.router.t(), TOPK, loss_coef=0.01)
        d_router = layer.router_gradient(h, routing, torch.zeros_like(y))
    print(f"balance loss {before:.6f} -> {float(routing.loss):.6f} after 20 steps")
    return before, float(routing.loss)


if __name__ == "__main__":
    main()
