"""Gradients of the feed-forward example's gradients are refused, not left out; a kept graph gives the same again."""
import os
import sys

import pytest

torch = pytest.importorskip("torch")

from tests.linear_util import rows

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("train", [False, True])
def test_gradients_of_gradients_are_refused(train):
    import feed_forward as ff
    block = ff.random_block(128, 96, train=train)
    x = rows(3, 20, 128).contiguous().requires_grad_()
    y = block(x)
    with pytest.raises(RuntimeError, match="no gradients of gradients"):
        torch.autograd.grad(y, x, torch.ones_like(y), create_graph=True)
    first = torch.autograd.grad(y, x, torch.ones_like(y), retain_graph=True)
    assert torch.equal(first[0], torch.autograd.grad(y, x, torch.ones_like(y))[0])
