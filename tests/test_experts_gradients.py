"""The expert operators have no backward pass: a call that autograd would
have to follow is refused, not answered with a result cut off from its inputs
(no GPU is needed for these checks)."""
import pytest

import block_scaled_mxfp4_bf16_amd as mx


def calls(torch):
    bf16 = dict(dtype=torch.bfloat16)
    Bw, Bs = torch.zeros((2, 64 * 16), dtype=torch.uint8), torch.zeros((2, 256 * 8), dtype=torch.uint8)
    off = torch.zeros(3, dtype=torch.int32)
    x, y, w, logits = torch.zeros((6, 64), **bf16), torch.zeros((8, 16), **bf16), torch.zeros((4, 2)), torch.zeros((4, 8))
    bias, res = torch.zeros(8), torch.zeros((4, 16), **bf16)
    ids = torch.zeros(6, dtype=torch.int32)
    return [
        (x, lambda: mx.gemv(x, Bw, Bs, 32, ids=ids)),
        (x, lambda: mx.gemm_grouped(x, Bw, Bs, off, 32)),
        (logits, lambda: mx.moe_route(logits, 2)),
        (bias, lambda: mx.moe_route(logits, 2, bias=bias)),
        (y, lambda: mx.moe_combine(y, w)),
        (w, lambda: mx.moe_combine(y, w)),
        (res, lambda: mx.moe_combine(y, w, residual=res)),
    ]


@pytest.mark.parametrize("i", range(7))
def test_inputs_that_require_gradients_are_refused(i):
    torch = pytest.importorskip("torch")
    t, call = calls(torch)[i]
    t.requires_grad_(True)
    with pytest.raises(RuntimeError, match="gradient"):
        call()
    with torch.no_grad(), pytest.raises(ValueError, match="cuda"):  # goes on to the next check
        call()
    t.requires_grad_(False)
    with pytest.raises(ValueError, match="cuda"):
        call()
