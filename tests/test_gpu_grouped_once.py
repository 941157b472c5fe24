"""mxfp4_gemm_grouped with a few rows of many large matrices, whose weights go
past the caches: against the product in 64 bits of a few of the groups, and the
same bits as each group alone."""
import numpy as np
import pytest

import block_scaled_mxfp4_bf16_amd as mx
from tests.expert_util import assert_within, dequant, product_limit
from tests.gpu_util import bf16_dev_to_bits, torch_cuda
from tests.test_gpu_grouped import activations, offsets_of, quantized
import oracle

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("N,K", [(4096, 1056), (2080, 2080)])
def test_few_rows_of_many_matrices(N, K, gated):
    torch = torch_cuda()
    E = 64
    assert E * N * (K // 2) >= 96 << 20
    g = torch.Generator(device="cuda")
    g.manual_seed(N)
    B = (torch.randn((E, N, K), generator=g, device="cuda") * K**-0.5).to(torch.bfloat16)
    Bw, Bs = mx.prepare_experts(B)
    sizes = np.random.default_rng(K).integers(0, 8, E)
    sizes[[0, 5, 40, 63]] = [0, 17, 33, 1]
    A = activations(torch, 1, int(sizes.sum()), K)
    C = mx.gemm_grouped(A, Bw, Bs, offsets_of(torch, sizes), N, gated=gated)
    at = np.concatenate([[0], np.cumsum(sizes)])
    a = quantized(A)
    for e in (1, 5, 40, 62, 63):
        lo, hi = int(at[e]), int(at[e + 1])
        w = dequant(*oracle.quantize(bf16_dev_to_bits(B[e].contiguous())))
        assert_within(C[lo:hi], *product_limit(a[lo:hi], w, "bf16", gated), "group %d" % e)
    for e in range(E):
        lo, hi = int(at[e]), int(at[e + 1])
        if hi > lo:
            assert torch.equal(C[lo:hi], mx.gemm_grouped(A[lo:hi], Bw[e], Bs[e], offsets_of(torch, [hi - lo]), N, gated=gated))
