"""The embedding's gradient added to what is there: numbers below 2^-126 count, and rows of either type may start anywhere."""

import pytest
import torch

from reduction_reducer_gb300 import embed_backward, layer_norm

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
KINDS = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _device():
    torch.cuda.set_device(0)


def draw(n, dim, kind, seed, extra=0, shift=0):
    """n rows, `extra` elements apart, from `shift` elements behind a 256-byte boundary on."""
    flat = torch.randn(n * (dim + extra) + shift, generator=torch.Generator("cuda").manual_seed(seed), device="cuda")
    return flat.to(KINDS[kind])[shift:].as_strided((n, dim), (dim + extra, 1))


@pytest.mark.parametrize("dim", [5, 16, 264])
@pytest.mark.parametrize("words", [9, 40, 3000])
def test_small_numbers_are_added(words, dim):
    """Whole multiples of 2^-149, of which every sum is exact: many tokens a row, few, and rows longer than a part."""
    gen = torch.Generator("cuda").manual_seed(dim)
    tokens = torch.randint(words, (700,), generator=gen, device="cuda")
    steps = torch.randint(-40, 41, (700, dim), generator=gen, device="cuda")
    there = torch.randint(-40, 41, (words, dim), generator=gen, device="cuda")
    grad, out = (t.double().mul(2.0 ** -149).float() for t in (steps, there))
    assert bool((grad.double() == steps * 2.0 ** -149).all())
    embed_backward(grad, tokens, out, accumulate=True)
    want = there.clone().index_add_(0, tokens, steps)
    assert bool((out.double() == want * 2.0 ** -149).all())


@pytest.mark.parametrize("dim", [7, 24, 520])
def test_additions_of_any_size(dim):
    """A token a row: one fp32 addition each, of numbers from 2^-149 to 2^-98 whose sums are exact in 64 bits, some of
    them nearly or quite each other's opposites, and zeros; rows of ordinary numbers beside them."""
    gen = torch.Generator("cuda").manual_seed(dim)

    def numbers():
        size = torch.exp2(-149 + 51 * torch.rand(600, dim, generator=gen, device="cuda", dtype=torch.float64))
        return (size * (1 - 2 * (torch.rand(600, dim, generator=gen, device="cuda") < 0.5))).float()

    grad, there = numbers(), numbers()
    pick = torch.rand(600, dim, generator=gen, device="cuda")
    there = torch.where(pick < 0.2, -grad, torch.where(pick < 0.4, -grad * (1 + 2.0 ** -20), there))
    grad[pick > 0.8] = 0.0
    there[(pick > 0.75) & (pick < 0.85)] = 0.0
    grad[:50], there[:50] = torch.randn(50, dim, generator=gen, device="cuda"), 0.0
    grad[60:70, dim // 2] = 0.0
    grad[70, 0], grad[71, 0], there[72, 0] = float("nan"), float("inf"), float("inf")
    want = (grad.double() + there.double()).float()
    order = torch.randperm(600, generator=gen, device="cuda")
    got = embed_backward(grad[order].contiguous(), order, there.clone(), accumulate=True)
    assert torch.allclose(got, want, rtol=0, atol=0, equal_nan=True)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("shift,extra", [(0, 4), (4, 0), (4, 8), (8, 4), (1, 0), (2, 6), (3, 3)])
def test_rows_that_start_anywhere(shift, extra, kind):
    """fp32 rows that gradients of either type are added to; nothing between the rows or around them is written."""
    n, dim = 37, 264
    tokens = torch.randint(-1, n + 1, (100,), generator=torch.Generator("cuda").manual_seed(1), device="cuda")
    grad, onto = draw(100, dim, kind, 2, extra, shift), draw(n, dim, "f32", 3)
    want = embed_backward(grad.contiguous(), tokens, onto.clone(), accumulate=True)
    assert not torch.equal(want, onto)
    whole = torch.full((n * (dim + extra) + shift,), 7.0, device="cuda")
    out = whole[shift:].as_strided((n, dim), (dim + extra, 1))
    out.copy_(onto)
    embed_backward(grad, tokens, out, accumulate=True)
    assert torch.equal(out, want)
    out.fill_(7.0)
    assert bool((whole == 7.0).all())


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("shift,extra", [(0, 4), (4, 0), (4, 8), (8, 4), (1, 0), (2, 6), (3, 3)])
@pytest.mark.parametrize("dim", [264, 1500, 17000])
def test_a_norm_writes_its_rows_alone(dim, shift, extra, kind):
    n = 9
    x = draw(n, dim, kind, shift, extra, shift)
    whole = torch.full((n * (dim + extra) + shift,), 7.0, dtype=x.dtype, device="cuda")
    out = whole[shift:].as_strided((n, dim), (dim + extra, 1))
    layer_norm(x, out=out)
    assert bool((out != 7.0).any())
    out.fill_(7.0)
    assert bool((whole == 7.0).all())
