"""A mixture-of-experts block on the expert operators: prompts and single tokens.

    python examples/moe_block.py [--experts 64] [--choices 8] [--hidden 2048] [--inner 2048] [--prompt 4096] [--batch 4]

builds a block with random weights, runs one prompt and some decoding steps
(captured into a graph, as a serving loop would), and prints the time of each.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import block_scaled_mxfp4_bf16_amd as mx  # noqa: E402


class MoEBlock:
    """y = x + sum over a token's experts of w * down(silu(gate(x)) * up(x)), weights in MXFP4.

    router [E, H], up [E, 2 * I, H] (the gate's rows first) and down [E, H, I]
    are bf16 cuda tensors; they are prepared once and not kept.  H and I have
    to be multiples of 32."""

    # Up to this many tokens a call reads each chosen expert for itself, with
    # unquantized activations; beyond, rows are sorted by expert and quantized.
    few = 4

    def __init__(self, router, up, down, choices, score="softmax", bias=None):
        self.router, self.choices, self.score, self.bias = router, choices, score, bias
        self.experts, self.hidden, self.inner = up.shape[0], up.shape[2], down.shape[2]
        self.up, self.down = mx.prepare_experts(up), mx.prepare_experts(down)

    def __call__(self, x):
        """x [T, H] bf16 -> [T, H] bf16, on the current stream; the host waits for nothing."""
        k = self.choices
        logits = x @ self.router.t()
        ids, weights, offsets, rows, pos = mx.moe_route(logits, k, score=self.score, bias=self.bias)
        if x.shape[0] <= self.few:
            h = mx.gemv(x, *self.up, 2 * self.inner, ids=ids, repeat=k, gated=True)
            y = mx.gemv(h, *self.down, self.hidden, ids=ids)
            return mx.moe_combine(y, weights, residual=x)
        h = mx.gemm_grouped(x, *self.up, offsets, 2 * self.inner, rows=rows, repeat=k, gated=True)
        y = mx.gemm_grouped(h, *self.down, offsets, self.hidden)
        return mx.moe_combine(y, weights, pos=pos, residual=x)


def random_block(experts, hidden, inner, choices, seed=0, **options):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape):
        return (torch.randn(shape, generator=g, device="cuda") * shape[-1] ** -0.5).to(torch.bfloat16)

    return MoEBlock(normal(experts, hidden), normal(experts, 2 * inner, hidden), normal(experts, hidden, inner), choices,
                    **options)


def time_us(call, n=20):
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
    for name, value in (("experts", 64), ("choices", 8), ("hidden", 2048), ("inner", 2048), ("prompt", 4096), ("batch", 4)):
        ap.add_argument("--" + name, type=int, default=value)
    a = ap.parse_args()
    block = random_block(a.experts, a.hidden, a.inner, a.choices)
    x = torch.randn((a.prompt, a.hidden), device="cuda").to(torch.bfloat16)
    us = time_us(lambda: block(x))
    print("prompt of %d tokens: %.1f us, %.2f M tokens/s" % (a.prompt, us, a.prompt / us))

    token = torch.randn((a.batch, a.hidden), device="cuda").to(torch.bfloat16)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):  # creates the workspaces of this stream
        block(token)
    stream.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        out = block(token)
    us = time_us(graph.replay, 100)
    print("decoding %d tokens: %.1f us a step, finite: %s" % (a.batch, us, bool(torch.isfinite(out).all())))


if __name__ == "__main__":
    main()
