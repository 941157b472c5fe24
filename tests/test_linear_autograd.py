"""What autograd is told of the dense layer's calls: tensors that they would cut
off from their gradients or tangents are refused, written ones count as changed
(no GPU is needed; the library is stood in for where a call gets that far)."""
import pytest

torch = pytest.importorskip("torch")

import block_scaled_mxfp4_bf16_amd as mx


def cpu(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


BW, BS = cpu(2, 512, dtype=torch.uint8), cpu(8, 256, dtype=torch.uint8)  # [32, 64], prepared

# name -> (tensors by name, call of them); those in WRITTEN are written
CALLS = {
    "linear": (lambda: dict(x=cpu(4, 64), bias=cpu(32), residual=cpu(4, 32), pre=cpu(4, 32), out=cpu(4, 32)),
               lambda t: mx.linear(t["x"], BW, BS, 32, bias=t["bias"], residual=t["residual"], pre=t["pre"], out=t["out"])),
    "pre": (lambda: dict(dy=cpu(4, 32), pre=cpu(4, 32), bias=cpu(32, dtype=torch.float32), out=cpu(4, 32)),
            lambda t: mx.linear_grad_pre(t["dy"], t["pre"], activation="silu", bias=t["bias"], out=t["out"])),
    "input": (lambda: dict(dz=cpu(4, 32), out=cpu(4, 64)), lambda t: mx.linear_grad_input(t["dz"], BW, BS, 64, out=t["out"])),
    "weight": (lambda: dict(dz=cpu(4, 32), x=cpu(4, 64), out=cpu(32, 64)),
               lambda t: mx.linear_grad_weight(t["dz"], t["x"], out=t["out"])),
}
WRITTEN = {"linear": ("pre", "out"), "pre": ("bias", "out"), "input": ("out",), "weight": ("out",)}
EACH = [(name, t) for name, (make, _) in CALLS.items() for t in make()]


@pytest.mark.parametrize("name,which", EACH)
def test_tensors_that_require_gradients_are_refused(name, which):
    make, call = CALLS[name]
    t = make()
    t[which].requires_grad_(True)
    with pytest.raises(RuntimeError, match="%s requires gradients" % which):
        call(t)
    with torch.no_grad(), pytest.raises(ValueError, match="cuda"):  # goes on to the next check
        call(t)


@pytest.mark.parametrize("name,which", EACH)
def test_tensors_with_a_tangent_are_refused(name, which):
    make, call = CALLS[name]
    t = make()
    with torch.autograd.forward_ad.dual_level():
        with pytest.raises(ValueError, match="cuda"):  # none has one
            call(t)
        t[which] = torch.autograd.forward_ad.make_dual(t[which], torch.ones_like(t[which]))
        assert not t[which].requires_grad
        with pytest.raises(RuntimeError, match="%s carries a forward-mode tangent" % which):
            call(t)
        with torch.no_grad(), pytest.raises(RuntimeError, match="%s carries a forward-mode tangent" % which):
            call(t)


class Library:
    """Takes every call and does nothing."""
    status = 0

    def __getattr__(self, name):
        return lambda *a: self.status


@pytest.fixture
def library(monkeypatch):
    mx._start()
    stand_in = Library()
    monkeypatch.setattr(mx, "_lib", stand_in)
    monkeypatch.setattr(mx, "_on_gpu", lambda dev: None)
    monkeypatch.setattr(mx, "_current_stream", lambda: 0)
    monkeypatch.setattr(mx, "_prepared", lambda *a: 1)
    return stand_in


@pytest.mark.parametrize("name", CALLS)
def test_written_tensors_count_as_changed(name, library):
    make, call = CALLS[name]
    t = make()
    before = {k: v._version for k, v in t.items()}
    call(t)
    for k, v in t.items():
        assert v._version - before[k] == (1 if k in WRITTEN[name] else 0), k
    with torch.inference_mode():  # tensors that keep no count
        call(make())


@pytest.mark.parametrize("write", [
    lambda kept: mx.linear(cpu(4, 64), BW, BS, 32, residual=kept, out=kept),
    lambda kept: mx.linear(cpu(4, 64), BW, BS, 32, pre=kept),
    lambda kept: mx.linear_grad_pre(cpu(4, 32), kept, activation="silu", out=kept),
])
def test_a_backward_pass_that_saved_a_written_tensor_says_so(write, library):
    w = torch.ones((4, 32), dtype=torch.bfloat16, requires_grad=True)
    kept = torch.full((4, 32), 2.0, dtype=torch.bfloat16)
    y = (w * kept).sum()
    write(kept)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()
