"""The mixture-of-experts example block: each stage against 64 bits from the
inputs that it really had, the whole against its stages, and its graphs."""
import importlib.util
import os

import numpy as np
import pytest

import block_scaled_mxfp4_bf16_amd as mx
import oracle
from tests.expert_util import HALF_STEP, assert_within, dequant, product_limit
from tests.gpu_util import bf16_dev_to_bits, torch_cuda

pytestmark = pytest.mark.gpu


def example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "moe_block.py")
    spec = importlib.util.spec_from_file_location("moe_block", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def weights(torch, seed, E, H, I):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    make = lambda *s: (torch.randn(s, generator=g, device="cuda") * s[-1] ** -0.5).to(torch.bfloat16)
    return make(E, H), make(E, 2 * I, H), make(E, H, I)


def values(t):
    """f64 values of bf16 matrices once quantized."""
    return [dequant(*oracle.quantize(bf16_dev_to_bits(m.contiguous()))) for m in t]


def products(rows, experts, w, is_gated):
    ref, lim = zip(*(product_limit(rows[i:i + 1], w[e], "bf16", is_gated) for i, e in enumerate(experts)))
    return np.concatenate(ref), np.concatenate(lim)


@pytest.mark.parametrize("T", [1, 4, 5, 70])
@pytest.mark.parametrize("score,with_bias", [("softmax", False), ("sigmoid", True)])
def test_stages_and_whole(T, score, with_bias):
    torch = torch_cuda()
    E, H, I, k = 6, 96, 160, 3
    router, up, down = weights(torch, T, E, H, I)
    bias = torch.linspace(-0.2, 0.2, E, device="cuda") if with_bias else None
    block = example().MoEBlock(router, up, down, k, score=score, bias=bias)
    x = torch.randn((T, H), device="cuda").to(torch.bfloat16)
    out = block(x)

    logits = x @ router.t()
    ids, w, offsets, rows, pos = mx.moe_route(logits, k, score=score, bias=bias)
    e_of = ids.cpu().numpy().reshape(-1)
    vup, vdown = values(up), values(down)
    if T <= block.few:
        h = mx.gemv(x, *block.up, 2 * I, ids=ids, repeat=k, gated=True)
        y = mx.gemv(h, *block.down, H, ids=ids)
        xin, hin, order = x.double().cpu().numpy(), h.double().cpu().numpy(), np.arange(T * k)
    else:
        h = mx.gemm_grouped(x, *block.up, offsets, 2 * I, rows=rows, repeat=k, gated=True)
        y = mx.gemm_grouped(h, *block.down, offsets, H)
        xin, hin = values([x])[0], values([h])[0]
        order = rows.cpu().numpy()
    assert_within(h, *products(xin[order // k], e_of[order], vup, True), "up")
    assert_within(y, *products(hin, e_of[order], vdown, False), "down")
    place = np.argsort(order).reshape(T, k)
    yv, wv = y.double().cpu().numpy(), w.double().cpu().numpy()
    terms = yv[place] * wv[:, :, None]
    ref = terms.sum(1) + x.double().cpu().numpy()
    # k + 1 f32 additions and k products, rounded once
    err = (2 * k + 1) * 2.0**-24 * (np.abs(terms).sum(1) + np.abs(x.double().cpu().numpy()))
    assert_within(out, ref, err + HALF_STEP["bf16"] * (np.abs(ref) + err), "sum")


def test_both_paths_agree_up_to_the_quantized_rows():
    """Rows that MXFP4 holds exactly make both paths' first product the same sum."""
    torch = torch_cuda()
    E, H, I, k, T = 4, 64, 64, 2, 4
    router, up, down = weights(torch, 1, E, H, I)
    block = example().MoEBlock(router, up, down, k)
    x = torch.tensor([0.5, -1.0, 3.0, 4.0], device="cuda").repeat(T, H // 4).to(torch.bfloat16)
    ids, _, offsets, rows, pos = mx.moe_route(x @ router.t(), k)
    few = mx.gemv(x, *block.up, 2 * I, ids=ids, repeat=k, gated=True)
    many = mx.gemm_grouped(x, *block.up, offsets, 2 * I, rows=rows, repeat=k, gated=True)[pos.reshape(-1).long()]
    ref, lim = products(x.double().cpu().numpy()[np.arange(T * k) // k], ids.cpu().numpy().reshape(-1), values(up), True)
    assert_within(few, ref, lim, "few")
    assert_within(many, ref, lim, "many")


@pytest.mark.parametrize("T", [2, 200])
def test_captured_into_a_graph(T):
    torch = torch_cuda()
    block = example().random_block(8, 128, 96, 2)
    x = torch.randn((T, 128), device="cuda").to(torch.bfloat16)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        block(x)
    stream.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        out = block(x)
    for i in range(4):
        x.copy_(torch.randn((T, 128), device="cuda").to(torch.bfloat16))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, block(x)), i
