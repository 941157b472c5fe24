"""A call on a stream other than torch's current one takes the memory of its
outputs from that stream: memory of the current stream could still be in use
there, and would be handed out again, when the output is dropped, to work that
does not wait for the call.  Nor is a dropped output handed out again before
what the current stream does with it is done."""
import pytest

import block_scaled_mxfp4_bf16_amd as mx
from tests.expert_util import Weights
from tests.gpu_util import torch_cuda

pytestmark = pytest.mark.gpu


def stream_of(torch, t):
    """Handle of the stream whose memory a tensor lies in."""
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= t.data_ptr() < seg["address"] + seg["total_size"]:
            return seg["stream"]
    raise AssertionError("not in torch's memory")


def calls(torch):
    E, N, K, T, k = 4, 64, 64, 200, 2
    w = Weights(torch, 1, E, N, K)
    B = torch.randn((E, N, K), device="cuda").to(torch.bfloat16)
    x = torch.randn((T, K), device="cuda").to(torch.bfloat16)
    logits = torch.randn((T, E), device="cuda")
    weights = torch.rand((T, k), device="cuda")
    offsets = torch.tensor([0, 40, 40, 90, T], dtype=torch.int32, device="cuda")
    q, s = mx.quantize(B[0])
    xq, xs = mx.quantize(x, shuffled_scales=True)
    y = torch.randn((T * k, N), device="cuda")
    torch.cuda.synchronize()
    return dict(
        quantize=lambda st: mx.quantize(x, stream=st),
        quantize_shuffled=lambda st: mx.quantize(x, shuffled_scales=True, stream=st),
        preshuffle_b=lambda st: mx.preshuffle_b(q, s, stream=st),
        prepare_b=lambda st: mx.prepare_b(B[0], stream=st),
        prepare_experts=lambda st: mx.prepare_experts(B, stream=st),
        gemm=lambda st: (mx.gemm(x, w.Bw[0], w.Bs[0], N, stream=st),),
        gemm_q=lambda st: (mx.gemm_q(xq, xs, w.Bw[0], w.Bs[0], N, stream=st),),
        gemv=lambda st: (mx.gemv(x, w.Bw[0], w.Bs[0], N, stream=st),),
        gemm_grouped=lambda st: (mx.gemm_grouped(x, w.Bw, w.Bs, offsets, N, stream=st),),
        moe_route=lambda st: mx.moe_route(logits, k, stream=st),
        moe_combine=lambda st: (mx.moe_combine(y, weights, stream=st),),
    )


NAMES = ["quantize", "quantize_shuffled", "preshuffle_b", "prepare_b", "prepare_experts", "gemm", "gemm_q", "gemv",
         "gemm_grouped", "moe_route", "moe_combine"]


@pytest.mark.parametrize("name", NAMES)
def test_outputs_lie_in_the_memory_of_their_stream(name):
    torch = torch_cuda()
    call = calls(torch)[name]
    here = call(None)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        there = call(stream)
        torch.cuda.synchronize()
        for a, b in zip(here, there):
            assert torch.equal(a, b)
            assert stream_of(torch, a) == torch.cuda.current_stream().cuda_stream
            assert stream_of(torch, b) == side.cuda_stream
    with torch.cuda.stream(side):  # the default stream, named by its handle, while another is current
        for b in call(0):
            assert stream_of(torch, b) == 0
        for b in call(None):
            assert stream_of(torch, b) == side.cuda_stream
    torch.cuda.synchronize()


@pytest.mark.parametrize("name", NAMES)
def test_a_dropped_output_is_not_overwritten_while_the_current_stream_reads_it(name):
    torch = torch_cuda()
    call = calls(torch)[name]
    side = torch.cuda.Stream()
    a = torch.randn((4096, 4096), device="cuda")
    b = torch.empty_like(a)
    torch.mm(a, a, out=b)
    torch.cuda.synchronize()
    out = call(side)
    torch.cuda.current_stream().wait_stream(side)
    places = {t.data_ptr() for t in out}
    done = torch.cuda.Event()
    for _ in range(100):  # tens of milliseconds of work on the current stream
        torch.mm(a, a, out=b)
    done.record()
    del out
    again = call(side)
    assert not done.query()
    assert not places & {t.data_ptr() for t in again}
    torch.cuda.synchronize()
