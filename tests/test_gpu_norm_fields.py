"""Layer norms whose gradient fields are given for one parameter alone, or for one that takes no gradient."""

import pytest
import torch

from reduction_reducer_gb300 import layer_norm, layer_norm_backward, layer_normed

pytestmark = pytest.mark.gpu

DIM = 40


@pytest.fixture(scope="module", autouse=True)
def _device():
    torch.cuda.set_device(0)


def draw(*shape, seed):
    return torch.randn(*shape, generator=torch.Generator("cuda").manual_seed(seed), device="cuda")


def expected(x, w, b, g):
    stats = layer_norm(x, w, b)[1]
    return layer_norm_backward(g, x, stats, w, torch.empty(DIM, device="cuda"), torch.empty(DIM, device="cuda"))


@pytest.mark.parametrize("fields", [(1, 0), (0, 1), (1, 1), (0, 0)])
@pytest.mark.parametrize("trained", [(1, 1), (1, 0), (0, 1), (0, 0)])
@pytest.mark.parametrize("input_grad", [True, False])
def test_each_gradient_goes_to_its_field_or_to_autograd(fields, trained, input_grad):
    x, g = draw(6, DIM, seed=1).requires_grad_(input_grad), draw(6, DIM, seed=2)
    params = [draw(DIM, seed=3 + i).requires_grad_(bool(on)) for i, on in enumerate(trained)]
    into = tuple(torch.ones(DIM, device="cuda") if on else None for on in fields)
    want = expected(x.detach(), *(p.detach() for p in params), g)
    y = layer_normed(x, *params, grad_into=into)
    if not (input_grad or any(trained)):
        assert not y.requires_grad
        return
    y.backward(g)
    assert (x.grad is not None) == input_grad and (not input_grad or torch.equal(x.grad, want[0]))
    for p, field, on, right in zip(params, into, trained, want[1:]):
        if field is not None:
            assert p.grad is None and torch.equal(field, 1 + right if on else torch.ones_like(field))
        elif on:
            assert torch.equal(p.grad, right)
        else:
            assert p.grad is None


def test_fields_without_a_parameter_stay():
    x, fields = draw(6, DIM, seed=1).requires_grad_(True), tuple(torch.ones(DIM, device="cuda") for _ in range(2))
    layer_normed(x, grad_into=fields).sum().backward()
    assert x.grad is not None and all(bool((f == 1).all()) for f in fields)
