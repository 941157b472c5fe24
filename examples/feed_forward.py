"""A gated feed-forward block on MXFP4 weights that gradients flow through.

    python examples/feed_forward.py [--hidden 4096] [--inner 8192] [--tokens 4096] [--train]

builds a block with random weights and prints the time of a forward and a
backward pass, and of a single token.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import block_scaled_mxfp4_bf16_amd as mx  # noqa: E402


class _Block(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, up, down, block):
        h, z = mx.linear(x, *block.prepared_up, 2 * block.inner, activation=block.activation, gated=True, pre=True)
        ctx.save_for_backward(x, h, z)
        ctx.block = block
        ctx.matrices = block.prepared_up, block.prepared_down  # those of this pass: prepare() makes new ones
        return mx.linear(h, *block.prepared_down, block.hidden, residual=x)

    @staticmethod
    def backward(ctx, dy):
        if torch.is_grad_enabled():  # create_graph: what is returned would be cut off from x without a word
            raise RuntimeError("the block has no gradients of gradients")
        x, h, z = ctx.saved_tensors
        block, dy = ctx.block, dy.contiguous()
        up, down = ctx.matrices
        dx = d_up = d_down = None
        if ctx.needs_input_grad[2]:
            d_down = mx.linear_grad_weight(dy, h, out_dtype=block.down.dtype)
        if ctx.needs_input_grad[0] or ctx.needs_input_grad[1]:
            dh = mx.linear_grad_input(dy, *down, block.inner)
            dz = mx.linear_grad_pre(dh, z, activation=block.activation, gated=True)
        if ctx.needs_input_grad[0]:
            dx = mx.linear_grad_input(dz, *up, block.hidden) + dy
        if ctx.needs_input_grad[1]:
            d_up = mx.linear_grad_weight(dz, x, out_dtype=block.up.dtype)
        return dx, d_up, d_down, None


class FeedForward(torch.nn.Module):
    """y = x + down(f(gate(x)) * up(x)), weights in MXFP4, activations quantized on the way.

    up [2 * I, H] (the gate's rows first) and down [H, I] are cuda tensors, H and I
    multiples of 32.  With train they are kept as parameters and have gradients,
    straight through the quantization; prepare() is then called after each step of
    the optimizer.  Otherwise only x has one, and only the prepared weights are kept."""

    def __init__(self, up, down, activation="silu", train=False):
        super().__init__()
        self.hidden, self.inner, self.activation = down.shape[0], down.shape[1], activation
        self.up = torch.nn.Parameter(up) if train else None
        self.down = torch.nn.Parameter(down) if train else None
        self.prepare(up, down)

    @torch.no_grad()
    def prepare(self, up=None, down=None):
        up, down = (self.up, self.down) if up is None else (up, down)
        self.prepared_up = mx.prepare_b(up.to(torch.bfloat16).contiguous())
        self.prepared_down = mx.prepare_b(down.to(torch.bfloat16).contiguous())

    def forward(self, x):
        """x [T, H] bf16 with contiguous rows -> [T, H] bf16."""
        return _Block.apply(x, self.up, self.down, self)


def random_block(hidden, inner, seed=0, **options):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda") * shape[-1] ** -0.5

    return FeedForward(normal(2 * inner, hidden), normal(hidden, inner), **options)


def time_us(call, n=10):
    call()
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    begin.record()
    for _ in range(n):
        call()
    end.record()
    end.synchronize()
    return begin.elapsed_time(end) * 1000 / n


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    for name, value in (("hidden", 4096), ("inner", 8192), ("tokens", 4096)):
        ap.add_argument("--" + name, type=int, default=value)
    ap.add_argument("--train", action="store_true", help="weights with gradients, too")
    a = ap.parse_args()
    block = random_block(a.hidden, a.inner, train=a.train)
    x = torch.randn((a.tokens, a.hidden), device="cuda").to(torch.bfloat16).requires_grad_()
    dy = torch.randn((a.tokens, a.hidden), device="cuda").to(torch.bfloat16)

    def step():
        block.zero_grad()
        x.grad = None
        block(x).backward(dy)

    with torch.no_grad():
        forward = time_us(lambda: block(x))
        token = time_us(lambda: block(x[:1]), 100)
    both = time_us(step)
    print("%d tokens: forward %.0f us, forward and backward %.0f us; one token: %.1f us; finite: %s" % (
        a.tokens, forward, both, token, bool(torch.isfinite(x.grad).all())))


if __name__ == "__main__":
    main()
