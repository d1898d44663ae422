"""A seed on the device that changes between dropout and its gradient: other elements would be dropped, so it is an error."""

import pytest
import torch

from reduction_reducer_gb300 import drop, dropped

pytestmark = pytest.mark.gpu


def test_a_seed_that_changed_is_refused():
    torch.cuda.set_device(0)
    x = torch.ones(4, 50, device="cuda", requires_grad=True)
    seed = torch.tensor([5], device="cuda")
    y = dropped(x, 0.4, seed, 3)
    y.sum().backward()
    assert torch.equal(x.grad, drop(torch.ones_like(x), 0.4, 5, 3))
    first, second = dropped(x, 0.4, seed, 3), dropped(x, 0.4, seed, 4)
    seed.add_(1)
    for y in (first, second):
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            y.sum().backward()
    # a copy for each pass may go on
    x.grad = None
    y = dropped(x, 0.4, seed.clone(), 3)
    seed.add_(1)
    y.sum().backward()
    assert torch.equal(x.grad, drop(torch.ones_like(x), 0.4, 6, 3))
