"""The feed-forward example: its gradients against the formulas, and that it runs."""
import os
import subprocess
import sys

import pytest

torch = pytest.importorskip("torch")

import block_scaled_mxfp4_bf16_amd as mx
from tests.expert_util import HALF_STEP
from tests.linear_util import act, act_error, assert_within, quantized, rounded, rows, sum_error

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))

pytestmark = pytest.mark.gpu


def prepared_values(w):
    """f64 values of prepare_b's result, by the same quantization of rows."""
    return quantized(w.detach().to(torch.bfloat16))


@pytest.mark.parametrize("tokens,hidden,inner", [(1, 64, 96), (40, 256, 160), (300, 512, 1024)])
@pytest.mark.parametrize("activation", ["silu", "gelu"])
def test_gradients(tokens, hidden, inner, activation):
    import feed_forward as ff
    block = ff.random_block(hidden, inner, activation=activation, train=True)
    x = rows(1, tokens, hidden).contiguous().requires_grad_()
    dy = rows(2, tokens, hidden, "bf16", 0.1).contiguous()
    block(x).backward(dy)
    up, down = prepared_values(block.up), prepared_values(block.down)
    # what the forward pass kept: the same bits, as every call of one size gives them
    with torch.no_grad():
        h, z = mx.linear(x.detach(), *block.prepared_up, 2 * inner, activation=activation, gated=True, pre=True)
    g, u = z[:, :inner].double(), z[:, inner:].double()
    f, slope = act(activation, g)
    ef, es = act_error(activation, g)
    d = dy.double()
    dh = d @ down
    edh = rounded(dh, sum_error(d, down.t().contiguous()), "bf16")  # dh is stored in bf16
    dz = torch.cat([dh * u * slope, dh * f], 1)
    edz = torch.cat([edh * (u * slope).abs() + (dh.abs() + edh) * u.abs() * es, edh * f.abs() + (dh.abs() + edh) * ef], 1)
    edz = rounded(dz, edz + 2.0**-22 * dz.abs(), "bf16")  # and so is dz
    dx = dz @ up
    edx = edz @ up.abs() + sum_error(dz.abs() + edz, up.t().contiguous())
    edx = rounded(dx, edx, "bf16")
    assert_within(x.grad, (dx + d, edx + HALF_STEP["bf16"] * ((dx + d).abs() + edx)), "dx")
    qx, qh = quantized(x.detach()), quantized(h)
    d_up, e_up = dz.t() @ qx, edz.t() @ qx.abs() + sum_error(dz.abs().t() + edz.t(), qx.t().contiguous())
    assert_within(block.up.grad, (d_up, e_up + 2.0**-23 * d_up.abs()), "gradient of up")
    d_down = d.t() @ qh
    assert_within(block.down.grad, (d_down, sum_error(d.t().contiguous(), qh.t().contiguous()) + 2.0**-23 * d_down.abs()),
                  "gradient of down")


def test_frozen_weights_and_changed_ones():
    import feed_forward as ff
    block = ff.random_block(128, 96)
    assert not list(block.parameters())
    x = rows(3, 20, 128).contiguous().requires_grad_()
    block(x).sum().backward()
    assert bool(torch.isfinite(x.grad).all())
    trained = ff.random_block(128, 96, train=True)
    y = trained(x)
    with torch.no_grad():
        assert torch.equal(y, block(x))
        trained.up.mul_(2)
    trained.prepare()
    before = x.grad.clone()
    x.grad = None
    y.sum().backward()  # with the weights of its own forward pass
    assert torch.equal(x.grad, before)
    assert not torch.equal(trained(x), y)


def test_runs_as_a_program():
    out = subprocess.run([sys.executable, os.path.join(ROOT, "examples", "feed_forward.py"), "--hidden", "512", "--inner",
                          "768", "--tokens", "300", "--train"], capture_output=True, text=True, timeout=100)
    assert out.returncode == 0, out.stderr[-2000:]
    assert "finite: True" in out.stdout
