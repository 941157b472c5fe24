"""mxfp4_gemv with more row tiles than one grid dimension holds."""
import numpy as np
import pytest

import block_scaled_mxfp4_bf16_amd as mx
from tests.expert_util import Weights, assert_within, product_limit
from tests.gpu_util import torch_cuda

pytestmark = pytest.mark.gpu


def test_one_matrix_per_row():
    torch = torch_cuda()
    M, N, K, E = 70001, 32, 64, 3
    w = Weights(torch, 1, E, N, K)
    r = np.random.default_rng(2)
    x = torch.from_numpy(r.standard_normal((M, K)).astype(np.float32)).to(torch.bfloat16).cuda()
    ids = r.integers(0, E, M).astype(np.int32)
    y = mx.gemv(x, w.Bw, w.Bs, N, ids=torch.from_numpy(ids).cuda(), out_dtype=torch.float32)
    xd = x.double().cpu().numpy()
    for e in range(E):
        ref, limit = product_limit(xd[ids == e], w.values[e], "f32", False)
        assert_within(y[torch.from_numpy(ids == e).cuda()], ref, limit, "matrix %d" % e)


def test_one_matrix():
    torch = torch_cuda()
    M, N, K = 1 << 20, 16, 32
    w = Weights(torch, 3, 1, N, K)
    x = torch.randn((M, K), device="cuda").to(torch.bfloat16)
    y = mx.gemv(x, w.Bw, w.Bs, N, out_dtype=torch.float32)
    ref, limit = product_limit(x.double().cpu().numpy(), w.values[0], "f32", False)
    assert_within(y, ref, limit, "all rows")


def test_no_rows():
    torch = torch_cuda()
    w = Weights(torch, 4, 1, 32, 32)
    assert mx.gemv(torch.empty((0, 32), device="cuda"), w.Bw, w.Bs, 32).shape == (0, 32)
