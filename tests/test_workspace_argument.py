"""gemm_grouped and moe_route take a workspace of the caller's: what they
refuse (no GPU is needed for these checks)."""
import inspect

import pytest

import block_scaled_mxfp4_bf16_amd as mx


def test_is_an_argument():
    for f in (mx.gemm_grouped, mx.moe_route):
        assert inspect.signature(f).parameters["workspace"].default is None


def test_refuses_one_that_is_none():
    torch = pytest.importorskip("torch")
    A = torch.zeros((6, 64), dtype=torch.bfloat16)
    Bw, Bs = torch.zeros((2, 64 * 16), dtype=torch.uint8), torch.zeros((2, 256 * 8), dtype=torch.uint8)
    off = torch.zeros(3, dtype=torch.int32)
    for bad in (torch.zeros((64, 64), dtype=torch.uint8)[:, ::2], torch.zeros(64, dtype=torch.uint8, device="meta")):
        with pytest.raises(ValueError, match="workspace"):
            mx.gemm_grouped(A, Bw, Bs, off, 32, workspace=bad)
        with pytest.raises(ValueError, match="workspace"):
            mx.moe_route(torch.zeros((4, 8)), 2, workspace=bad)
