"""mxfp4_gemv over the whole range of scale bytes: both ends are exact for
every type of x, weights of 2^128 and more, which no 16- or 32-bit type holds, among
them; and f32 rows count in steps of 2^-133."""
import numpy as np
import pytest

import block_scaled_mxfp4_bf16_amd as mx
import oracle
from tests.expert_util import assert_within, dequant, dtype_of, product_limit
from tests.gpu_util import torch_cuda

pytestmark = pytest.mark.gpu

N, K, M = 48, 416, 5

# bf16 and f32 rows take a group of scale byte 253 twice and of 254 four times,
# with the largest scale that bf16 has room for: up to four times the additions,
# so four times the error of an f32 sum.
TIMES = 4


def prepared(torch, q, s):
    return torch.from_numpy(oracle.preshuffle_b(q)).cuda(), torch.from_numpy(oracle.shuffle_scales(s, N, K)).cuda()


def codes(r, largest):
    """Random codes of magnitude number up to `largest`, both signs."""
    c = r.integers(0, largest + 1, (N, K)) | (r.integers(0, 2, (N, K)) << 3)
    return (c[:, 0::2] | (c[:, 1::2] << 4)).astype(np.uint8)


# the largest code whose weight is below 2^128: 6 up to byte 252, 3 at 253, 1.5 at 254
@pytest.mark.parametrize("byte,largest", [(0, 7), (1, 7), (2, 7), (3, 7), (127, 7), (252, 7), (253, 5), (254, 3)])
@pytest.mark.parametrize("xt", ["bf16", "f16", "f32"])
def test_every_scale(xt, byte, largest):
    torch = torch_cuda()
    r = np.random.default_rng(byte)
    q, s = codes(r, largest), np.full((N, K // 32), byte, np.uint8)
    # rows that bring the sums near 1 as far as their type reaches
    top = 14 if xt == "f16" else 100
    x = r.standard_normal((M, K)) * 2.0 ** min(top, max(-top, 127 - byte))
    x = torch.from_numpy(x.astype(np.float32)).to(dtype_of(torch, xt)).cuda()
    ref, limit = product_limit(x.double().cpu().numpy(), dequant(q, s), "f32", False)
    y = mx.gemv(x, *prepared(torch, q, s), N, out_dtype=torch.float32)
    assert_within(y, ref, limit * (TIMES if byte > 252 else 1), "%s, scale byte %d" % (xt, byte))


@pytest.mark.parametrize("xt", ["bf16", "f16", "f32"])
def test_scales_of_both_ends_in_one_row(xt):
    torch = torch_cuda()
    r = np.random.default_rng(5)
    q, s = codes(r, 3), r.choice(np.array([0, 1, 2, 125, 128, 252, 253, 254], np.uint8), (N, K // 32))
    x = torch.from_numpy((r.standard_normal((M, K)) * 2.0**-10).astype(np.float32)).to(dtype_of(torch, xt)).cuda()
    ref, limit = product_limit(x.double().cpu().numpy(), dequant(q, s), "f32", False)
    assert_within(mx.gemv(x, *prepared(torch, q, s), N, out_dtype=torch.float32), ref, TIMES * limit, xt)


@pytest.mark.parametrize("xt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("byte,smallest", [(253, 6), (254, 4)])
def test_weights_beyond_f32(byte, smallest, xt):
    torch = torch_cuda()
    r = np.random.default_rng(byte)
    c = r.integers(smallest, 8, (N, K))
    q, s = (c[:, 0::2] | (c[:, 1::2] << 4)).astype(np.uint8), np.full((N, K // 32), byte, np.uint8)
    x = (r.standard_normal((M, K)) * 2.0**-20).astype(np.float32)
    x[:, ::3] = 0
    x = torch.from_numpy(x).to(dtype_of(torch, xt)).cuda()
    ref, limit = product_limit(x.double().cpu().numpy(), dequant(q, s), "f32", False)
    assert_within(mx.gemv(x, *prepared(torch, q, s), N, out_dtype=torch.float32), ref, TIMES * limit, xt)


@pytest.mark.parametrize("xt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("gated,M", [(False, 1), (False, 17), (True, 3)])
def test_single_groups_of_large_weights(xt, gated, M):
    """One step in the middle has them, the others have not; more column tiles than one."""
    torch = torch_cuda()
    r = np.random.default_rng(8)
    n, k = 2112, 1120
    c = r.integers(0, 16, (n, k))
    q, s = (c[:, 0::2] | (c[:, 1::2] << 4)).astype(np.uint8), np.full((n, k // 32), 130, np.uint8)
    s[r.integers(0, n, 40), r.integers(0, k // 32, 40)] = 253
    s[r.integers(0, n, 40), r.integers(0, k // 32, 40)] = 254
    x = r.standard_normal((M, k)) * (2.0**-22 if xt == "f16" else 2.0**-70)
    x = torch.from_numpy(x.astype(np.float32)).to(dtype_of(torch, xt)).cuda()
    w = dequant(q, s)
    if gated:  # ordinary gates, so that the product says something of both halves
        w[:n // 2] = np.where(np.abs(w[:n // 2]) > 1e6, 0, w[:n // 2])
        q[:n // 2][np.repeat(s[:n // 2] > 200, 16, axis=1)] = 0
    bw = torch.from_numpy(oracle.preshuffle_b(q)).cuda(), torch.from_numpy(oracle.shuffle_scales(s, n, k)).cuda()
    ref, limit = product_limit(x.double().cpu().numpy(), w, "f32", gated)
    assert_within(mx.gemv(x, *bw, n, gated=gated, out_dtype=torch.float32), ref, TIMES * limit, xt)


def test_f32_rows_count_in_steps():
    """Elements below 2^-110 keep what lies on the steps of 2^-133."""
    torch = torch_cuda()
    r = np.random.default_rng(6)
    q, s = codes(r, 7), np.full((N, K // 32), 127 + 60, np.uint8)
    w = dequant(q, s)
    for e in (-100, -109, -115, -125, -130):
        x = torch.from_numpy((r.standard_normal((M, K)) * 2.0**e).astype(np.float32)).cuda()
        ref, limit = product_limit(x.double().cpu().numpy(), w, "f32", False)
        # 24 bits from 2^-110 on are whole steps
        limit = limit + 2.0**-133 * np.abs(w).sum(1)[None]
        assert_within(mx.gemv(x, *prepared(torch, q, s), N), ref, limit, "2^%d" % e)


@pytest.mark.parametrize("xt", ["bf16", "f16", "f32"])
def test_a_scale_of_no_number_touches_its_columns_only(xt):
    torch = torch_cuda()
    r = np.random.default_rng(9)
    q, s = codes(r, 7), np.full((N, K // 32), 127, np.uint8)
    s[5, 3] = s[17, 12] = s[40, 0] = 255
    x = torch.from_numpy(r.standard_normal((M, K)).astype(np.float32)).to(dtype_of(torch, xt)).cuda()
    y = mx.gemv(x, *prepared(torch, q, s), N, out_dtype=torch.float32)
    assert not bool(torch.isfinite(y[:, [5, 17, 40]]).any())
    rest = [n for n in range(N) if n not in (5, 17, 40)]
    ref, limit = product_limit(x.double().cpu().numpy(), dequant(q, s)[rest], "f32", False)
    assert_within(y[:, rest], ref, limit, xt)
