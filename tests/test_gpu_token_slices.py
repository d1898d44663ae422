"""Tokens and targets as slices of one batch, which is how a next-token loss has them."""

import pytest
import torch

from reduction_reducer_gb300 import embed, embed_backward, embedded, logprobs, logprobs_backward, scored

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    torch.cuda.set_device(0)


@pytest.mark.parametrize("bits", [torch.int32, torch.int64])
@pytest.mark.parametrize("side", [False, True])
def test_slices_are_what_they_are_a_copy_of(bits, side):
    gen = torch.Generator("cuda").manual_seed(0)
    text = torch.randint(-1, 31, (5, 13), generator=gen, device="cuda").to(bits)
    table, grad = (torch.randn(*s, generator=gen, device="cuda") for s in ((31, 24), (5, 12, 24)))
    logits = torch.randn(5, 12, 31, generator=gen, device="cuda")
    one = torch.ones(5, 12, device="cuda")
    tokens, targets = text[:, :-1], text[:, 1:]
    assert not tokens.is_contiguous() and not targets.is_contiguous()
    stream = torch.cuda.Stream() if side else None
    torch.cuda.synchronize()

    def run(tokens, targets):
        got = logprobs(logits, targets, 3, entropy=True, stream=stream)
        out = [embed(table, tokens, stream=stream),
               embed_backward(grad, tokens, torch.empty(31, 24, device="cuda"), stream=stream), *got,
               logprobs_backward(one, logits, targets, got.stats, stream=stream)]
        torch.cuda.synchronize()
        return out

    for a, b in zip(run(tokens, targets), run(tokens.contiguous(), targets.contiguous())):
        assert torch.equal(a, b)


def test_under_autograd():
    gen = torch.Generator("cuda").manual_seed(0)
    text = torch.randint(31, (4, 9), generator=gen, device="cuda")
    table = torch.randn(31, 16, generator=gen, device="cuda", requires_grad=True)

    def grad(tokens, targets):
        return torch.autograd.grad(scored(embedded(table, tokens) @ table.detach().t(), targets).logp.sum(), table)[0]

    assert torch.equal(grad(text[:, :-1], text[:, 1:]), grad(text[:, :-1].contiguous(), text[:, 1:].contiguous()))


def test_a_place_without_a_next_token_is_left_out():
    """The logits of all places, with a target outside of the vocabulary in the last: those of the others, uncopied.  Rows of
    31 start at other places of 16 bytes in the copy, so their sums have another order: with u = 2^-24, |log p| below 16
    and log S below 16, each is off by (250 + 2 log S + 4 |log p| + 4 |log p + log S|) u < 500 u at most."""
    gen = torch.Generator("cuda").manual_seed(0)
    text = torch.randint(31, (4, 9), generator=gen, device="cuda")
    logits = torch.randn(4, 9, 31, generator=gen, device="cuda")
    with pytest.raises(ValueError, match="one distance"):
        logprobs(logits[:, :-1], text[:, 1:])
    targets = torch.nn.functional.pad(text[:, 1:], (0, 1), value=-1)
    got, want = logprobs(logits, targets).logp, logprobs(logits[:, :-1].contiguous(), text[:, 1:].contiguous()).logp
    assert bool((want.abs() < 16).all()) and bool((logits.abs() < 8).all())
    assert torch.allclose(got[:, :-1], want, rtol=0, atol=1000 * 2.0 ** -24) and not bool(got[:, -1].any())
