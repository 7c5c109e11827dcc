"""A gated feed-forward block trained in 16 bits and served in 4, from this
package's operators:

    python examples/ffn_layer.py [--tokens T] [--act silu|gelu|gelu_tanh]

    training: h = act(x Wg^T) * (x Wu^T)   gated_linear, gated_linear_backward
              y = h Wd^T                   torch's product
    serving:  both weights to 4 bits       w4_quant
              h and y of any batch         w4_gated_linear, w4_linear
Random weights; the sizes are small.
"""
import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import block_scaled_fp8_act_amd as fb  # noqa: E402

HIDDEN, INTER = 1024, 2816


class GatedLinear(torch.autograd.Function):
    """gated_linear and its gradients, for what of x and w asks for one."""

    @staticmethod
    def forward(ctx, x, w, act):
        ctx.act = act
        if not any(ctx.needs_input_grad[:2]):
            return fb.gated_linear(x, w, act)
        h, factors = fb.gated_linear(x, w, act, save=True)
        ctx.save_for_backward(x, w, factors)
        return h

    @staticmethod
    def backward(ctx, d_h):
        x, w, factors = ctx.saved_tensors
        need_x, need_w, _ = ctx.needs_input_grad
        return *fb.gated_linear_backward(d_h.contiguous(), x, w, factors, ctx.act, need_x, need_w), None


class Block:
    """The block's weights: gate rows first, then the ups', and the down projection."""

    def __init__(self, act="silu", device="cuda", seed=0):
        g = torch.Generator(device=device).manual_seed(seed)
        rand = lambda n, k: (torch.randn(n, k, device=device, generator=g) * k ** -0.5).bfloat16()  # noqa: E731
        self.act = act
        self.up, self.down = rand(2 * INTER, HIDDEN).requires_grad_(), rand(HIDDEN, INTER).requires_grad_()

    def forward(self, x):
        return GatedLinear.apply(x, self.up, self.act) @ self.down.t()

    def in_4_bits(self, group=64):
        """The block as it is served: y of x."""
        up, down = (fb.w4_quant(w.detach(), group, zeros=True) for w in (self.up, self.down))
        return lambda x: fb.w4_linear(fb.w4_gated_linear(x, *up, act=self.act), *down)


def main(argv=None):
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("--tokens", type=int, default=500)
    p.add_argument("--act", choices=list(fb.ACTS), default="silu")
    a = p.parse_args(argv)
    block = Block(a.act)
    g = torch.Generator(device="cuda").manual_seed(1)
    x, want = (torch.randn(a.tokens, HIDDEN, device="cuda", generator=g).bfloat16() for _ in range(2))
    for step in range(3):
        loss = (block.forward(x) - want).float().square().mean()
        loss.backward()
        print(f"step {step}: loss {float(loss.detach()):.4f}")
        with torch.no_grad():
            for w in (block.up, block.down):
                w -= 0.5 * w.grad
                w.grad = None
    with torch.no_grad():
        y, served = block.forward(x), block.in_4_bits()
        off = (served(x) - y).float().norm() / y.float().norm()
    one = served(x[:1])
    print(f"served {a.tokens} tokens in 4 bits: {float(off):.3f} of the 16-bit block's output apart; one token "
          f"alone: largest difference {float((one - served(x)[:1]).abs().max()):.4f}")
    return float(off)


if __name__ == "__main__":
    main()
