"""The dense layer against its 64-bit form, over sizes, types, activations, strides and ways of calling."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import block_scaled_mxfp4_bf16_amd as mx
from tests.expert_util import dtype_of
from tests.linear_util import ACTS, Matrix, assert_within, linear_limit, rows

pytestmark = pytest.mark.gpu

SIZES = [(1, 16, 32), (1, 4096, 1024), (2, 48, 96), (5, 2112, 704), (15, 32, 4096), (16, 96, 160), (17, 512, 64),
         (31, 160, 1056), (33, 64, 128), (63, 224, 512), (64, 1024, 256), (65, 336, 288), (127, 128, 992), (129, 4096, 64),
         (200, 112, 2080), (257, 576, 416), (300, 1040, 1024), (513, 272, 160), (1000, 768, 224), (1025, 2064, 96)]


def check(M, N, K, activation, gated, y_type, bias, residual, seed):
    w = Matrix(seed, N, K)
    x = rows(seed + 1, M, K)
    b = (torch.randn(N, device="cuda") * 0.3).to(dtype_of(torch, bias)) if bias else None
    r = rows(seed + 2, M, N // 2 if gated else N, y_type) if residual else None
    want_y, want_z = linear_limit(x, w.values, y_type, b, activation, gated, r)
    y, z = mx.linear(x, w.Bw, w.Bs, N, bias=b, activation=activation, gated=gated, residual=r, pre=True,
                     out_dtype=dtype_of(torch, y_type))
    assert_within(z, want_z, "pre")
    assert_within(y, want_y, "y")
    # without keeping z
    assert torch.equal(y, mx.linear(x, w.Bw, w.Bs, N, bias=b, activation=activation, gated=gated, residual=r,
                                    out_dtype=dtype_of(torch, y_type)))


@pytest.mark.parametrize("i,size", enumerate(SIZES))
def test_sizes(i, size):
    M, N, K = size
    check(M, N, K, ACTS[i % 5], False, ["bf16", "f32", "f16"][i % 3], ["", "bf16", "f32", "f16"][i % 4], i % 2 == 0, 10 * i)


@pytest.mark.parametrize("i,size", enumerate(s for s in SIZES if s[1] % 32 == 0))
def test_gated_sizes(i, size):
    M, N, K = size
    check(M, N, K, ACTS[(i + 2) % 5], True, ["f32", "bf16", "f16"][i % 3], ["f32", "", "bf16", "f16"][i % 4], i % 2 == 1,
          10 * i + 5)


@pytest.mark.parametrize("M", [3, 40, 333])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("activation", ACTS)
def test_activations(activation, gated, M):
    check(M, 320, 288, activation, gated, "f32", "f32", True, M)


@pytest.mark.parametrize("activation", ACTS)
def test_far_arguments(activation):
    """Pre-activations that a bias pushes far out, where exponentials and cubes overflow."""
    w = Matrix(3, 64, 64)
    x = rows(4, 8, 64)
    for far in (0.0, 1.0, 12.0, 40.0, 300.0, 1e5, 1e15, 1e30):
        for sign in (1, -1):
            b = torch.full((64,), sign * far, device="cuda")
            want, _ = linear_limit(x, w.values, "f32", b, activation)
            y = mx.linear(x, w.Bw, w.Bs, 64, bias=b, activation=activation, out_dtype=torch.float32)
            assert_within(y, want, "%s at %g" % (activation, sign * far))


def guarded(M, cols, dtype, left, right):
    """A tensor of rows inside longer rows of a value that nothing else holds."""
    whole = torch.full((M + 2, left + cols + right), 777.0, dtype=dtype, device="cuda")
    return whole, whole[1:M + 1, left:left + cols]


@pytest.mark.parametrize("M", [1, 7, 50, 270])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("left,right", [(8, 8), (1, 2), (4, 5)])
def test_strides_and_what_lies_around(left, right, gated, M):
    N, K = 160, 224
    cols = N // 2 if gated else N
    w = Matrix(1, N, K)
    x = rows(2, M, K, pad=24)
    for y_type in ("bf16", "f32"):
        dtype = dtype_of(torch, y_type)
        r = rows(3, M, cols, y_type, pad=right)
        whole_y, y = guarded(M, cols, dtype, left, right)
        whole_z, z = guarded(M, N, torch.bfloat16, left, right)
        want_y, want_z = linear_limit(x, w.values, y_type, None, "gelu", gated, r)
        got = mx.linear(x, w.Bw, w.Bs, N, activation="gelu", gated=gated, residual=r, pre=z, out=y)
        assert got[0] is y and got[1] is z
        assert_within(y, want_y, "y")
        assert_within(z, want_z, "pre")
        for whole, part in ((whole_y, y), (whole_z, z)):
            kept = whole.clone()
            part.fill_(777.0)
            assert bool((whole == 777.0).all()), "something outside the rows was written"
            whole.copy_(kept)


@pytest.mark.parametrize("M", [1, 20, 400])
def test_residual_in_place(M):
    w = Matrix(5, 192, 96)
    x = rows(6, M, 96)
    stream = rows(7, M, 192)
    want, _ = linear_limit(x, w.values, "bf16", residual=stream.clone())
    assert mx.linear(x, w.Bw, w.Bs, 192, residual=stream, out=stream) is stream
    assert_within(stream, want, "y")


def test_no_rows():
    w = Matrix(5, 64, 32)
    x = torch.empty((0, 32), dtype=torch.bfloat16, device="cuda")
    y, z = mx.linear(x, w.Bw, w.Bs, 64, activation="silu", gated=True, pre=True)
    assert y.shape == (0, 32) and z.shape == (0, 64)


@pytest.mark.parametrize("M", [1, 9, 70, 520])
def test_same_bits_every_time_and_in_both_encoder_modes(M):
    w = Matrix(8, 1056, 1056)
    x = rows(9, M, 1056)
    first = mx.linear(x, w.Bw, w.Bs, 1056, activation="silu", gated=True)
    for _ in range(20):
        assert torch.equal(first, mx.linear(x, w.Bw, w.Bs, 1056, activation="silu", gated=True))
    mx.mxfp4_set_quant_mode(1)
    try:
        assert torch.equal(first, mx.linear(x, w.Bw, w.Bs, 1056, activation="silu", gated=True))
    finally:
        mx.mxfp4_set_quant_mode(0)


@pytest.mark.parametrize("M", [2, 100])
def test_scale_bytes_from_the_smallest_to_the_largest(M):
    """Weights whose scale bytes run from 0 to 250 in one matrix; sums are compared where f32 holds them."""
    def scales(r, s):
        return r.integers(0, 251, s.shape).astype(np.uint8)
    w = Matrix(11, 64, 128, scales=scales)
    x = rows(12, M, 128, scale=1.0)
    want, _ = linear_limit(x, w.values, "f32")
    y = mx.linear(x, w.Bw, w.Bs, 64, out_dtype=torch.float32)
    assert_within(y, want, "y")


@pytest.mark.parametrize("M", [3, 150])
def test_other_stream_and_own_workspace(M):
    N, K = 512, 256
    w = Matrix(13, N, K)
    x = rows(14, M, K)
    want = mx.linear(x, w.Bw, w.Bs, N, activation="relu")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    ws = torch.empty(mx.mxfp4_linear_workspace_bytes(M, N, K) + 256, dtype=torch.uint8, device="cuda")
    assert ws.data_ptr() % 256 == 0
    a = mx.linear(x, w.Bw, w.Bs, N, activation="relu", stream=side)
    b = mx.linear(x, w.Bw, w.Bs, N, activation="relu", stream=side, workspace=ws)
    side.synchronize()
    assert torch.equal(a, want) and torch.equal(b, want)
    need = mx.mxfp4_linear_workspace_bytes(M, N, K)
    if need:
        with pytest.raises(RuntimeError, match="workspace"):
            mx.linear(x, w.Bw, w.Bs, N, workspace=ws[:need - 1])


@pytest.mark.parametrize("M", [1, 30, 300])
def test_graph_replays(M):
    N, K = 384, 320
    w = Matrix(15, N, K)
    x = rows(16, M, K)
    y = torch.empty((M, N // 2), dtype=torch.bfloat16, device="cuda")
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        mx.linear(x, w.Bw, w.Bs, N, activation="gelu_tanh", gated=True, out=y)
    stream.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        mx.linear(x, w.Bw, w.Bs, N, activation="gelu_tanh", gated=True, out=y)
    for seed in range(4):
        x.copy_(rows(20 + seed, M, K))
        want = mx.linear(x, w.Bw, w.Bs, N, activation="gelu_tanh", gated=True)
        y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want)


def test_one_row_of_the_largest_k():
    w = Matrix(17, 32, 1 << 17)
    x = rows(18, 2, 1 << 17)
    want, _ = linear_limit(x, w.values, "f32")
    assert_within(mx.linear(x, w.Bw, w.Bs, 32, out_dtype=torch.float32), want, "y")
