"""The dense layer at sizes that make its large tiles: many rows, many columns, edges in every direction."""
import pytest

torch = pytest.importorskip("torch")

import block_scaled_mxfp4_bf16_amd as mx
from tests.expert_util import dtype_of
from tests.linear_util import ACTS, Matrix, assert_within, linear_limit, rows

pytestmark = pytest.mark.gpu

SIZES = [(8200, 1040, 224), (300, 32784, 96), (2100, 4112, 416), (4352, 2048, 512), (4161, 2112, 352), (513, 24640, 704),
         (8449, 1024, 32), (6000, 1600, 1056), (257, 16448, 160), (70000, 48, 64), (33, 33024, 544)]


def check(M, N, K, activation, gated, y_type, bias, residual, pre, seed, left=0):
    """With `left`, x, y, residual and pre lie in longer rows, y and pre from that column on."""
    w = Matrix(seed, N, K)
    x = rows(seed + 1, M, K, pad=8 * left)
    cols = N // 2 if gated else N
    b = (torch.randn(N, device="cuda") * 0.3).to(dtype_of(torch, bias)) if bias else None
    r = rows(seed + 2, M, cols, y_type, pad=left) if residual else None
    whole_y = torch.full((M + 1, cols + 2 * left), 777.0, dtype=dtype_of(torch, y_type), device="cuda")
    whole_z = torch.full((M + 1, N + 2 * left), 777.0, dtype=torch.bfloat16, device="cuda")
    y, z = whole_y[:-1, left:left + cols], whole_z[:-1, left:left + N]
    want_y, want_z = linear_limit(x, w.values, y_type, b, activation, gated, r)
    mx.linear(x, w.Bw, w.Bs, N, bias=b, activation=activation, gated=gated, residual=r, pre=z if pre else None, out=y)
    assert_within(y, want_y, "y")
    if pre:
        assert_within(z, want_z, "pre")
    again = torch.empty((M, cols), dtype=y.dtype, device="cuda")
    mx.linear(x, w.Bw, w.Bs, N, bias=b, activation=activation, gated=gated, residual=r, out=again)
    assert torch.equal(again, y)
    y.fill_(777.0)
    z.fill_(777.0)
    assert bool((whole_y == 777.0).all()) and bool((whole_z == 777.0).all()), "something outside the rows was written"


@pytest.mark.parametrize("i,size", enumerate(SIZES))
def test_sizes(i, size):
    check(*size, ACTS[i % 5], False, ["bf16", "f32", "f16"][i % 3], ["", "bf16", "f32", "f16"][i % 4], i % 2 == 0,
          i % 3 != 1, 100 * i)


@pytest.mark.parametrize("i,size", enumerate(s for s in SIZES if s[1] % 32 == 0))
def test_gated_sizes(i, size):
    check(*size, ACTS[(i + 2) % 5], True, ["bf16", "f32", "f16"][(i + 1) % 3], ["f32", "", "bf16", "f16"][i % 4],
          i % 2 == 1, i % 3 != 0, 100 * i + 50)


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("activation", ACTS)
def test_activations(activation, gated):
    check(2100, 4160, 160, activation, gated, "f32", "f32", True, True, 7)


@pytest.mark.parametrize("y_type", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("left", [1, 2, 4, 8])
@pytest.mark.parametrize("gated", [False, True])
def test_strides_and_what_lies_around(gated, left, y_type):
    check(2100, 4160, 96, "silu", gated, y_type, "bf16", True, True, 11, left)


def test_same_bits_every_time():
    w = Matrix(8, 4096, 1056)
    x = rows(9, 2500, 1056)
    first = mx.linear(x, w.Bw, w.Bs, 4096, activation="silu", gated=True)
    for _ in range(10):
        assert torch.equal(first, mx.linear(x, w.Bw, w.Bs, 4096, activation="silu", gated=True))
    plain = mx.linear(x, w.Bw, w.Bs, 4096)
    for _ in range(10):
        assert torch.equal(plain, mx.linear(x, w.Bw, w.Bs, 4096))


def test_other_weights_in_turn():
    """Layers of other sizes one after another on one workspace: nothing of one shows in the next."""
    layers = [(Matrix(i, N, K), rows(20 + i, M, K)) for i, (M, N, K) in enumerate([(2304, 4096, 512), (8200, 1040, 224), (40, 4096, 704)])]
    want = [mx.linear(x, w.Bw, w.Bs, w.N) for w, x in layers]
    for _ in range(3):
        for (w, x), y in zip(layers, want):
            assert torch.equal(y, mx.linear(x, w.Bw, w.Bs, w.N))


def test_residual_in_place():
    w = Matrix(5, 4112, 96)
    x = rows(6, 2100, 96)
    stream = rows(7, 2100, 4112)
    want, _ = linear_limit(x, w.values, "bf16", residual=stream.clone())
    assert mx.linear(x, w.Bw, w.Bs, 4112, residual=stream, out=stream) is stream
    assert_within(stream, want, "y")
