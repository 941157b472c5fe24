"""The gradient products in their 256 x 256 tiles over many stages of the sum: full and ragged tiles, every output type and store."""
import os
import re

import pytest

torch = pytest.importorskip("torch")

import block_scaled_mxfp4_bf16_amd as mx
from tests.expert_util import dtype_of
from tests.linear_util import Matrix, assert_within, product_limit, quantized, rows

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "block_scaled_mxfp4_bf16_amd", "csrc",
                      "grad_product.hip")

# Rows I and columns K of the output, length J of the sum.  A stage is 64 of J, a round of the loop three stages.
SIZES = [(4096, 3584, 1024), (4100, 3104, 1040), (4100, 3104, 2064), (2064, 8224, 208), (12304, 1056, 592), (6160, 2048, 80)]


def tiles256(I, K):
    return -(-I // 256) * -(-K // 256)


def test_the_sizes_take_256_x_256_tiles():
    with open(SOURCE) as f:
        (least,) = re.findall(r"if \(tiles < (\d+)\) \{\s*p\.form = Plan::kTile128", f.read())
    assert all(tiles256(I, K) >= int(least) and I > 128 for I, K, _ in SIZES + [OFFSETS])
    assert max(J for _, _, J in SIZES) > 10 * 3 * 64


def gapped(t, pad=8):
    """The same in longer rows, which hold NaN behind it, and a row of NaN after the last."""
    whole = torch.full((t.shape[0] + 1, t.shape[1] + pad), float("nan"), dtype=t.dtype, device="cuda")
    whole[:-1, :t.shape[1]] = t
    return whole[:-1, :t.shape[1]]


@pytest.mark.gpu
@pytest.mark.parametrize("t", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("i,size", enumerate(SIZES))
def test_input_gradient(i, size, t):
    I, K, J = size
    w = Matrix(i, J, K)
    dz = gapped(rows(10 + i, I, J, "bf16", 0.1))
    out = mx.linear_grad_input(dz, w.Bw, w.Bs, K, out_dtype=dtype_of(torch, t))
    assert_within(out, product_limit(dz, w.values, t), "dx")
    assert torch.equal(out, mx.linear_grad_input(dz, w.Bw, w.Bs, K, out_dtype=dtype_of(torch, t)))


@pytest.mark.gpu
@pytest.mark.parametrize("t", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("i,size", enumerate(SIZES))
def test_weight_gradient(i, size, t):
    I, K, J = size
    I, M = (I + 15) // 16 * 16, J + i % 3 * 5 - 5  # N is a multiple of 16, M need not be
    dz, x = gapped(rows(20 + i, M, I, "bf16", 0.1)), gapped(rows(30 + i, M, K))
    out = mx.linear_grad_weight(dz, x, out_dtype=dtype_of(torch, t))
    assert_within(out, product_limit(dz.t().contiguous(), quantized(x), t), "dw")
    assert torch.equal(out, mx.linear_grad_weight(dz, x, out_dtype=dtype_of(torch, t)))


OFFSETS = (4112, 3104, 272)


@pytest.mark.gpu
@pytest.mark.parametrize("t", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("left,right", [(8, 8), (1, 2), (4, 1)])
def test_what_lies_around(left, right, t):
    I, K, J = OFFSETS
    w = Matrix(1, J, K)
    dz, dzt, x = rows(2, I, J, "bf16", 0.1), rows(3, J, I, "bf16", 0.1), rows(4, J, K)
    for call, want in ((lambda o: mx.linear_grad_input(dz, w.Bw, w.Bs, K, out=o), product_limit(dz, w.values, t)),
                       (lambda o: mx.linear_grad_weight(dzt, x, out=o), product_limit(dzt.t().contiguous(), quantized(x), t))):
        whole = torch.full((I + 2, left + K + right), 777.0, dtype=dtype_of(torch, t), device="cuda")
        out = whole[1:-1, left:left + K]
        assert call(out) is out
        assert_within(out, want, "out")
        out.fill_(777.0)
        assert bool((whole == 777.0).all()), "something outside the rows was written"


@pytest.mark.gpu
def test_same_bits_every_time():
    """The ring of three stages and the two halves of T, rewritten many times: any order of the waves gives the same."""
    I, K, J = SIZES[2]
    w = Matrix(1, J, K)
    dz, dzt, x = rows(2, I, J, "bf16", 0.1), rows(3, J, (I + 15) // 16 * 16, "bf16", 0.1), rows(4, J, K)
    first = mx.linear_grad_input(dz, w.Bw, w.Bs, K), mx.linear_grad_weight(dzt, x)
    for _ in range(30):
        assert torch.equal(first[0], mx.linear_grad_input(dz, w.Bw, w.Bs, K))
        assert torch.equal(first[1], mx.linear_grad_weight(dzt, x))
