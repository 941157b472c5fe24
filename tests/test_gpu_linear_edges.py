"""The ends of the number ranges of the gradient products: scale bytes up to 255, and values that bf16 does not hold."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import block_scaled_mxfp4_bf16_amd as mx
from tests.linear_util import Matrix, assert_within, product_limit, quantized, rows

pytestmark = pytest.mark.gpu


def infinite(values):
    """Weights as grad_input takes them: those of 2^128 and more are infinite."""
    return torch.where(values.abs() >= 2.0**128, values.sign() * float("inf"), values)


@pytest.mark.parametrize("byte", [251, 252, 253, 254])
@pytest.mark.parametrize("M", [3, 140, 2100])
def test_input_gradient_of_the_largest_scale_bytes(M, byte):
    """One weight row of that byte, multiplied by a row of dz that is one there: its values, exact or infinite; and
    rows of dz that are zero there: NaN where the value is infinite, since it counts as such, and the others' sums elsewhere."""
    N, K = 64, 6144 if M > 2000 else 96  # the last in the largest tiles

    def scales(r, s):
        s[37] = byte
        return s
    w = Matrix(byte, N, K, scales=scales)
    big = infinite(w.values[37])
    assert bool(torch.isinf(big).any()) == (byte > 252) and bool(torch.isfinite(big).any())
    dz = rows(1, M, N, "bf16", 0.1)
    dz[:, 37] = 0
    dz[1] = 0
    dz[1, 37] = 1
    got = mx.linear_grad_input(dz, w.Bw, w.Bs, K, out_dtype=torch.float32)
    assert torch.equal(got[1].double(), big)
    lost = torch.isinf(big)
    rest = torch.arange(M, device="cuda") != 1
    assert bool(got[rest][:, lost].isnan().all())
    ref, limit = product_limit(dz, w.values, "f32")
    assert_within(got[rest][:, ~lost], (ref[rest][:, ~lost], limit[rest][:, ~lost]), "dx")


@pytest.mark.parametrize("M", [3, 140])
def test_input_gradient_of_scale_byte_255(M):
    """Stands for NaN: of its group of 32 columns only."""
    N, K = 64, 96

    def scales(r, s):
        s[37, 1] = 255
        return s
    w = Matrix(5, N, K, scales=scales)
    dz = rows(1, M, N, "bf16", 0.1)
    got = mx.linear_grad_input(dz, w.Bw, w.Bs, K, out_dtype=torch.float32)
    assert not bool(torch.isfinite(got[:, 32:64]).any())
    ref, limit = product_limit(dz, torch.nan_to_num(w.values, 0.0, 0.0, 0.0), "f32")
    keep = [k for k in range(K) if not 32 <= k < 64]
    assert_within(got[:, keep], (ref[:, keep], limit[:, keep]), "dx")


@pytest.mark.parametrize("M,N,K", [(5, 48, 96), (300, 48, 96), (70, 4096, 4096)])
def test_weight_gradient_of_the_largest_rows(M, N, K):
    """x that quantizes to 2^128 in one column: that column is infinite, or NaN where dz is 0; the largest values that
    bf16 holds, in the same group, and all other columns are as ever."""
    x, dz = rows(1, M, K), rows(2, M, N, "bf16", 0.1)
    x[2, 40], x[2, 41], x[2, 42] = 3.0e38, 2.9e38, -2.0e38
    dz[2, :8] = 0
    q = quantized(x)
    assert float(q[2, 40]) == 2.0**128 and float(q[2, 41]) == 3 * 2.0**126
    for mode in (0, 1):
        mx.mxfp4_set_quant_mode(mode)
        try:
            dw = mx.linear_grad_weight(dz, x)
        finally:
            mx.mxfp4_set_quant_mode(0)
        assert bool(dw[:8, 40].isnan().all())
        assert torch.equal(dw[8:, 40].double(), dz[2, 8:].double().sign() * float("inf"))
        ref, limit = product_limit(dz.t().contiguous(), torch.where(q.abs() >= 2.0**128, 0.0, q), "f32")
        keep = torch.arange(K, device="cuda") != 40
        assert_within(dw[:, keep], (ref[:, keep], limit[:, keep]), "dw")


@pytest.mark.parametrize("M,N,K", [(5, 48, 96), (300, 48, 96)])
def test_weight_gradient_of_the_smallest_rows(M, N, K):
    """x down to bf16's smallest subnormal, whose groups have scale byte 0, in f32 gradients that hold the products."""
    x = rows(1, M, K) * 2.0**-126
    x[0, 5] = 2.0**-133
    dz = rows(2, M, N, "bf16", 1.0) * 2.0**20
    assert float(quantized(x).abs().max()) < 2.0**-120
    dw = mx.linear_grad_weight(dz, x)
    assert bool((dw != 0).any())
    assert_within(dw, product_limit(dz.t().contiguous(), quantized(x), "f32"), "dw")
