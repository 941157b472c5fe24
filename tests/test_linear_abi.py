"""What the dense layer's entry points refuse; no GPU is needed, nothing is enqueued."""
import ctypes

import pytest

import block_scaled_mxfp4_bf16_amd as mx

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
P = 1 << 20  # an aligned address that nothing reads


def linear(**c):
    d = dict(x=P, ldx=64, B=P, S=P, bias=None, bias_type=0, act=0, gated=0, res=None, ld_res=0, y=P, y_type=0, ldy=32,
             pre=None, ld_pre=0, M=4, N=32, K=64, ws=P, ws_bytes=0)
    d.update(c)
    return mx.lib().mxfp4_linear(*[d[k] for k in (
        "x", "ldx", "B", "S", "bias", "bias_type", "act", "gated", "res", "ld_res", "y", "y_type", "ldy", "pre", "ld_pre",
        "M", "N", "K", "ws", "ws_bytes")], None)


def grad_pre(**c):
    d = dict(dy=P, t=0, ld_dy=32, pre=P, ld_pre=32, act=2, gated=0, dz=P, ld_dz=32, db=P, M=4, N=32, ws=P, ws_bytes=0)
    d.update(c)
    return mx.lib().mxfp4_linear_grad_pre(*[d[k] for k in (
        "dy", "t", "ld_dy", "pre", "ld_pre", "act", "gated", "dz", "ld_dz", "db", "M", "N", "ws", "ws_bytes")], None)


def grad_input(**c):
    d = dict(dz=P, ld_dz=4096, B=P, S=P, dx=P, t=0, ld_dx=64, M=4, N=4096, K=64, ws=P, ws_bytes=0)
    d.update(c)
    return mx.lib().mxfp4_linear_grad_input(*[d[k] for k in (
        "dz", "ld_dz", "B", "S", "dx", "t", "ld_dx", "M", "N", "K", "ws", "ws_bytes")], None)


def grad_weight(**c):
    d = dict(dz=P, ld_dz=32, x=P, ldx=64, dw=P, t=2, ld_dw=64, M=4, N=32, K=64, ws=P, ws_bytes=0)
    d.update(c)
    return mx.lib().mxfp4_linear_grad_weight(*[d[k] for k in (
        "dz", "ld_dz", "x", "ldx", "dw", "t", "ld_dw", "M", "N", "K", "ws", "ws_bytes")], None)


FAR = (1 << 20) + 8


@pytest.mark.parametrize("call,change,status", [
    (linear, dict(x=None), INVALID), (linear, dict(B=None), INVALID), (linear, dict(S=None), INVALID),
    (linear, dict(y=None), INVALID), (linear, dict(M=-1), INVALID), (linear, dict(N=0), INVALID),
    (linear, dict(K=0), INVALID), (linear, dict(act=5), INVALID), (linear, dict(act=-1), INVALID),
    (linear, dict(y_type=3), INVALID), (linear, dict(bias=P, bias_type=7), INVALID), (linear, dict(ldx=32), INVALID),
    (linear, dict(ldy=31), INVALID), (linear, dict(gated=1, ldy=15), INVALID), (linear, dict(res=P, ld_res=31), INVALID),
    (linear, dict(pre=P, ld_pre=31), INVALID), (linear, dict(x=P + 8), INVALID), (linear, dict(ldx=68), INVALID),
    (linear, dict(B=P + 4), INVALID), (linear, dict(S=P + 8), INVALID), (linear, dict(y=P + 1), INVALID),
    (linear, dict(y=P + 2, y_type=2), INVALID), (linear, dict(bias=P + 2, bias_type=2), INVALID),
    (linear, dict(res=P + 1, ld_res=32), INVALID), (linear, dict(pre=P + 1, ld_pre=32), INVALID),
    (linear, dict(K=48), UNSUPPORTED), (linear, dict(N=24, ldy=32), UNSUPPORTED),
    (linear, dict(N=48, ldy=48, gated=1), UNSUPPORTED), (linear, dict(M=(1 << 20) + 1), UNSUPPORTED),
    (linear, dict(N=(1 << 20) + 16, ldy=1 << 21), UNSUPPORTED), (linear, dict(K=(1 << 17) + 32, ldx=1 << 18), UNSUPPORTED),
    (linear, dict(N=1 << 17, K=1 << 15, ldx=1 << 15, ldy=1 << 17), UNSUPPORTED), (linear, dict(ldx=FAR), UNSUPPORTED),
    (linear, dict(ldy=FAR), UNSUPPORTED), (linear, dict(res=P, ld_res=FAR), UNSUPPORTED),
    (linear, dict(pre=P, ld_pre=FAR), UNSUPPORTED), (linear, dict(M=0, x=None, y=None), OK),
    (grad_pre, dict(dy=None), INVALID), (grad_pre, dict(dz=None), INVALID), (grad_pre, dict(pre=None), INVALID),
    (grad_pre, dict(pre=None, act=0, gated=1, ld_dy=16), INVALID), (grad_pre, dict(M=-1), INVALID),
    (grad_pre, dict(N=0), INVALID), (grad_pre, dict(act=9), INVALID), (grad_pre, dict(t=-1), INVALID),
    (grad_pre, dict(ld_dy=31), INVALID), (grad_pre, dict(ld_dz=31), INVALID), (grad_pre, dict(ld_pre=31), INVALID),
    (grad_pre, dict(dy=P + 2, t=2), INVALID), (grad_pre, dict(dz=P + 1), INVALID), (grad_pre, dict(db=P + 2), INVALID),
    (grad_pre, dict(pre=P + 1), INVALID), (grad_pre, dict(N=24), UNSUPPORTED), (grad_pre, dict(N=16, gated=1), UNSUPPORTED),
    (grad_pre, dict(M=(1 << 20) + 1), UNSUPPORTED), (grad_pre, dict(ld_dy=FAR), UNSUPPORTED),
    (grad_pre, dict(ld_dz=FAR), UNSUPPORTED), (grad_pre, dict(ld_pre=FAR), UNSUPPORTED),
    (grad_pre, dict(ws_bytes=1), WORKSPACE), (grad_pre, dict(ws=P + 128, ws_bytes=1 << 20), WORKSPACE),
    (grad_pre, dict(M=0, db=None, dy=None, dz=None, pre=None), OK),
    (grad_input, dict(dz=None), INVALID), (grad_input, dict(B=None), INVALID), (grad_input, dict(S=None), INVALID),
    (grad_input, dict(dx=None), INVALID), (grad_input, dict(M=-1), INVALID), (grad_input, dict(t=3), INVALID),
    (grad_input, dict(ld_dz=4095), INVALID), (grad_input, dict(ld_dx=63), INVALID), (grad_input, dict(dz=P + 8), INVALID),
    (grad_input, dict(ld_dz=4100), INVALID), (grad_input, dict(B=P + 8), INVALID), (grad_input, dict(dx=P + 2, t=2), INVALID),
    (grad_input, dict(K=40, ld_dx=64), UNSUPPORTED), (grad_input, dict(N=4088), UNSUPPORTED),
    (grad_input, dict(M=(1 << 20) + 1), UNSUPPORTED), (grad_input, dict(ld_dz=FAR), UNSUPPORTED),
    (grad_input, dict(ld_dx=FAR), UNSUPPORTED), (grad_input, dict(ws_bytes=1), WORKSPACE),
    (grad_input, dict(M=0, dz=None, dx=None), OK),
    (grad_weight, dict(dz=None), INVALID), (grad_weight, dict(x=None), INVALID), (grad_weight, dict(dw=None), INVALID),
    (grad_weight, dict(M=0, dw=None), INVALID), (grad_weight, dict(t=3), INVALID), (grad_weight, dict(ld_dz=31), INVALID),
    (grad_weight, dict(ldx=63), INVALID), (grad_weight, dict(ld_dw=63), INVALID), (grad_weight, dict(dz=P + 8), INVALID),
    (grad_weight, dict(x=P + 2), INVALID), (grad_weight, dict(ldx=68), INVALID), (grad_weight, dict(dw=P + 2), INVALID),
    (grad_weight, dict(K=48), UNSUPPORTED), (grad_weight, dict(N=24), UNSUPPORTED),
    (grad_weight, dict(M=(1 << 20) + 1), UNSUPPORTED), (grad_weight, dict(ld_dw=FAR), UNSUPPORTED),
    (grad_weight, dict(ldx=FAR), UNSUPPORTED), (grad_weight, dict(ld_dz=FAR), UNSUPPORTED),
    (grad_weight, dict(ws_bytes=1), WORKSPACE),
])
def test_refusals(call, change, status):
    assert call(**change) == status


def test_workspace_sizes():
    for f in (mx.mxfp4_linear_workspace_bytes, mx.mxfp4_linear_grad_input_workspace_bytes,
              mx.mxfp4_linear_grad_weight_workspace_bytes):
        assert f(0, 32, 64) == 0 and f(4, 24, 64) == 0 and f(4, 32, 48) == 0 and f(1 << 21, 32, 64) == 0
    assert mx.mxfp4_linear_grad_pre_workspace_bytes(0, 32) == 0
    # all of the largest sizes within 64 bits, and none less than what its data takes
    assert 0 < mx.mxfp4_linear_workspace_bytes(1 << 20, 1 << 14, 1 << 17) < 1 << 46
    assert mx.mxfp4_linear_grad_weight_workspace_bytes(1 << 20, 1 << 14, 1 << 17) >= (1 << 36) * 17 // 16


torch = pytest.importorskip("torch")


def cpu(*shape, dtype=torch.bfloat16, **kw):
    return torch.zeros(shape, dtype=dtype, **kw)


BW, BS = cpu(2, 512, dtype=torch.uint8), cpu(8, 256, dtype=torch.uint8)  # [32, 64], prepared


@pytest.mark.parametrize("call,error", [
    (lambda: mx.linear(cpu(4, 64), BW, BS, 32), "cuda tensors"),
    (lambda: mx.linear(cpu(4, 64, dtype=torch.float16), BW, BS, 32), "x must be bf16"),
    (lambda: mx.linear(cpu(64), BW, BS, 32), "M, K"),
    (lambda: mx.linear(cpu(64, 4).t(), BW, BS, 32), "contiguous rows"),
    (lambda: mx.linear(cpu(4, 64), BW, BS, 48), "prepared"),
    (lambda: mx.linear(cpu(4, 64), torch.cat([BW, BW]), torch.cat([BS, BS]), 32), "one matrix"),
    (lambda: mx.linear(cpu(4, 64), BW, BS, 32, activation="tanh"), "activation"),
    (lambda: mx.linear(cpu(4, 64), BW, BS, 32, bias=cpu(31)), "bias"),
    (lambda: mx.linear(cpu(4, 64), BW, BS, 32, bias=cpu(32, dtype=torch.int32)), "bf16, f16 or f32"),
    (lambda: mx.linear(cpu(4, 64), BW, BS, 32, residual=cpu(4, 31)), "residual"),
    (lambda: mx.linear(cpu(4, 64), BW, BS, 32, gated=True, residual=cpu(4, 32)), "residual"),
    (lambda: mx.linear(cpu(4, 64), BW, BS, 32, residual=cpu(4, 32), out_dtype=torch.float32), "residual is"),
    (lambda: mx.linear(cpu(4, 64), BW, BS, 32, pre=cpu(4, 16)), "pre"),
    (lambda: mx.linear(cpu(4, 64), BW, BS, 32, pre=cpu(4, 32, dtype=torch.float32)), "pre must be bf16"),
    (lambda: mx.linear(cpu(4, 64), BW, BS, 32, out=cpu(4, 33)), "out"),
    (lambda: mx.linear(cpu(4, 64, requires_grad=True), BW, BS, 32), "x requires gradients"),
    (lambda: mx.linear(cpu(4, 64), BW, BS, 32, bias=cpu(32, requires_grad=True)), "bias requires gradients"),
    (lambda: mx.linear(cpu(4, 64), BW, BS, 32, residual=cpu(4, 32, requires_grad=True)), "residual requires gradients"),
    (lambda: mx.linear_grad_pre(cpu(4, 32), None, activation="silu"), "needs pre"),
    (lambda: mx.linear_grad_pre(cpu(4, 32), None, gated=True), "needs pre"),
    (lambda: mx.linear_grad_pre(cpu(4, 32), cpu(4, 32), activation="silu", gated=True), "pre"),
    (lambda: mx.linear_grad_pre(cpu(4, 32), cpu(4, 32, dtype=torch.float32), activation="silu"), "pre must be bf16"),
    (lambda: mx.linear_grad_pre(cpu(4, 32), cpu(4, 32), out=cpu(4, 32, dtype=torch.float32)), "out must be bf16"),
    (lambda: mx.linear_grad_pre(cpu(4, 32, requires_grad=True), None), "dy requires gradients"),
    (lambda: mx.linear_grad_pre(cpu(4, 32), None, bias=cpu(32)), "bias"),
    (lambda: mx.linear_grad_pre(cpu(4, 32), None, bias=cpu(31, dtype=torch.float32)), "bias"),
    (lambda: mx.linear_grad_pre(cpu(4, 32), None), "cuda tensors"),
    (lambda: mx.linear_grad_input(cpu(4, 32), BW, BS, 96), "prepared"),
    (lambda: mx.linear_grad_input(cpu(4, 32, dtype=torch.float32), BW, BS, 64), "dz must be bf16"),
    (lambda: mx.linear_grad_input(cpu(4, 32), BW, BS, 64, out=cpu(4, 63)), "out"),
    (lambda: mx.linear_grad_input(cpu(4, 32), BW, BS, 64), "cuda tensors"),
    (lambda: mx.linear_grad_weight(cpu(4, 32), cpu(5, 64)), "x must have"),
    (lambda: mx.linear_grad_weight(cpu(4, 32), cpu(4, 64, dtype=torch.float32)), "x must be bf16"),
    (lambda: mx.linear_grad_weight(cpu(4, 32), cpu(4, 64), out=cpu(64, 32)), "out"),
    (lambda: mx.linear_grad_weight(cpu(4, 32), cpu(4, 64)), "cuda tensors"),
])
def test_tensor_functions_refuse(call, error):
    with pytest.raises((ValueError, TypeError, RuntimeError), match=error):
        call()


def test_signatures_take_64_bit_sizes():
    for name in ("mxfp4_linear", "mxfp4_linear_grad_pre", "mxfp4_linear_grad_input", "mxfp4_linear_grad_weight"):
        assert ctypes.c_int64 in getattr(mx.lib(), name).argtypes
