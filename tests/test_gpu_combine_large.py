"""mxfp4_moe_combine where the rows are too many to be kept in a cache: the same
bits as of a few tokens at a time, in place and with places of no row."""
import pytest

import block_scaled_mxfp4_bf16_amd as mx
from tests.gpu_util import torch_cuda

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("yt,ot", [("bfloat16", "bfloat16"), ("float32", "bfloat16"), ("float16", "float32")])
@pytest.mark.parametrize("T,k,N", [(4099, 8, 2048), (30011, 3, 1032), (1, 70000, 1024)])
def test_same_as_a_few_tokens_at_a_time(T, k, N, yt, ot):
    torch = torch_cuda()
    g = torch.Generator(device="cuda")
    g.manual_seed(T)
    y = torch.randn((T * k, N), generator=g, device="cuda").to(getattr(torch, yt))
    assert y.nbytes >= 96 << 20
    w = torch.rand((T, k), generator=g, device="cuda")
    pos = torch.randperm(T * k, generator=g, device="cuda").reshape(T, k).to(torch.int32)
    pos[::7, 0] = -1
    pos[T // 2, k - 1] = T * k
    res = torch.randn((T, N), generator=g, device="cuda").to(getattr(torch, ot))
    want = torch.empty_like(res)
    step = max(1, T // 16)
    for t in range(0, T, step):
        if T > 1:
            mx.moe_combine(y, w[t:t + step], pos=pos[t:t + step], residual=res[t:t + step], out=want[t:t + step])
    if T == 1:  # the same rows in a matrix whose stride keeps them off 16-byte loads
        wide = torch.empty((T * k, N + 1), dtype=y.dtype, device="cuda")
        wide[:, 1:] = y
        mx.moe_combine(wide[:, 1:], w, pos=pos, residual=res, out=want)
    got = res.clone()
    mx.moe_combine(y, w, pos=pos, residual=got, out=got)
    assert torch.equal(got, want)
    assert bool(torch.isfinite(got).all())
