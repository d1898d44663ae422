"""Edges of routing and its gradient on the GPU: confident experts, scales near fp32's least, softmax scores by their
definition whatever the batch, and every store path of the gradient."""

import numpy as np
import pytest
import torch

from oracle import route as R
from reduction_reducer_gb300 import route, route_backward

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
KINDS = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _device():
    torch.cuda.set_device(0)


def generator(seed):
    return torch.Generator("cuda").manual_seed(seed)

@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("renorm", [False, True])
def test_sigmoid_gradient_of_confident_experts(renorm, dtype):
    """Chosen logits of 8 to 20, where 1 - s is 3e-4 to 2e-9: its own relative error stays a few roundings (expf 4u, a
    sum and a quotient), those of the weights 64u, so as they are a gradient is within 80u of itself; renormalised it is
    a difference of terms of at most the row's sum of |g w|, which the factor 1 - s multiplies whole."""
    T, E, k, scale = 400, 32, 8, 2.5
    x = (torch.rand(T, E, generator=generator(1), device="cuda") * 12 + 8).to(KINDS[dtype])
    g = torch.randn(T, k, generator=generator(2), device="cuda")
    index, w = route(x, k, score="sigmoid", renorm=renorm, scale=scale)
    d = route_backward(g, x, index, w, score="sigmoid", renorm=renorm, scale=scale).double()
    at = index.long()
    z, gd = x.double().gather(1, at), g.double()
    s, rest = 1 / (1 + torch.exp(-z)), 1 / (1 + torch.exp(z))        # rest: 1 - s without a difference
    if renorm:
        share = s / s.sum(1, keepdim=True)
        want = scale * share * (gd - (gd * share).sum(1, keepdim=True)) * rest
        bound = 160 * U * (gd * share * scale).abs().sum(1, keepdim=True) * rest
    else:
        want = scale * gd * s * rest
        bound = 80 * U * want.abs()
    if dtype == "bf16":
        bound = bound + 2.0 ** -8 * want.abs()
    got = d.gather(1, at)
    assert bool(((got - want).abs() <= bound).all())
    assert int((d != 0).sum()) <= T * k

@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("scale", [1e-39, -3e-40])
def test_gradient_at_scales_below_the_least_normal_number(scale, score):
    """1 / scale is infinite in fp32.  Weights and products are subnormal, each within 2^-150 of itself: k + 4 of these
    beside the bound of ordinary scales."""
    T, E, k = 50, 24, 6
    x = torch.randn(T, E, generator=generator(3), device="cuda")
    g = torch.randn(T, k, generator=generator(4), device="cuda")
    index, w = route(x, k, score=score, renorm=True, scale=scale)
    assert bool((w != 0).all())
    d = route_backward(g, x, index, w, score=score, renorm=True, scale=scale).double().cpu().numpy()
    fp32_scale = float(np.float32(scale))
    for t in range(T):
        gt = g[t].double().cpu().numpy()
        want = R.backward_token(x[t].double().cpu().numpy(), index[t].tolist(), gt, score, True, fp32_scale)
        size = np.abs(gt * w[t].double().cpu().numpy()).sum()
        assert np.all(np.abs(d[t] - want) <= 160 * U * size + (k + 4) * 2.0 ** -149 * (1 + np.abs(gt).max())), t

def softmax_definition(x, groups):
    """Softmax scores in fp32, step by step: e = exp(x - largest); the sum of a group's experts eight by eight, one
    after another, the eights' sums and then the groups' in pairs; e over the sum."""
    T, E = x.shape
    x = x.float()
    e = torch.exp(x - x.amax(1, keepdim=True))
    size = E // groups
    eights = 1
    while 8 * eights < size:
        eights *= 2
    count = 1
    while count < groups:
        count *= 2
    wide = torch.zeros(T, count, 8 * eights, device="cuda")
    wide[:, :groups, :size] = e.view(T, groups, size)
    wide = wide.view(T, count * eights, 8)
    total = wide[:, :, 0]
    for j in range(1, 8):
        total = total + wide[:, :, j]
    while total.shape[1] > 1:
        total = total[:, 0::2] + total[:, 1::2]
    return e / total


def softmax_choice(x, k, bias, groups, top):
    """(indices, weights) of route(score="softmax", bias=bias) by the definition in fp32."""
    T, E = x.shape
    s = softmax_definition(x, groups)
    c = s + bias
    if groups > 1:
        worth = c.view(T, groups, E // groups).topk(min(2, E // groups)).values.sum(2)
        first = worth.argsort(dim=1, descending=True, stable=True)[:, :top]
        stay = torch.zeros(T, groups, dtype=torch.bool, device="cuda").scatter_(1, first, True)
        c = torch.where(stay.repeat_interleave(E // groups, dim=1), c, float("-inf"))
    index = c.argsort(dim=1, descending=True, stable=True)[:, :k]
    return index, s.gather(1, index)


# every layout: one to four eights a lane, groups that fill lanes and groups that do not, ones that fit no layout
SOFTMAX = [(8, 1, 1, 3), (24, 1, 1, 4), (60, 1, 1, 5), (128, 1, 1, 8), (200, 1, 1, 12), (256, 1, 1, 8), (512, 1, 1, 10),
           (64, 8, 3, 6), (72, 8, 3, 8), (60, 4, 2, 5), (256, 8, 4, 8), (320, 10, 3, 6), (500, 10, 4, 8), (510, 3, 2, 5),
           (510, 30, 7, 8), (512, 16, 4, 8)]


@pytest.mark.parametrize("E,groups,top,k", SOFTMAX)
@pytest.mark.parametrize("spread", [0.0, 6e-8, 1e-6, 1e-2])
def test_softmax_scores_and_near_ties_follow_the_definition(E, groups, top, k, spread):
    """A bias that brings the experts of a row within `spread` of one another, rows that differ by a shift (the same
    scores but for roundings) and rows of their own: choices and weights are the fp32 definition's bit for bit."""
    x = torch.randn(1, E, generator=generator(E), device="cuda") + torch.randn(60, 1, generator=generator(7), device="cuda")
    x[40:] = torch.randn(20, E, generator=generator(8), device="cuda") * 1.5
    bias = 0.7 - softmax_definition(x[:1], groups)[0] + torch.rand(E, generator=generator(9), device="cuda") * spread
    index, w = route(x, k, bias=bias, groups=groups, top_groups=top)
    want, weight = softmax_choice(x, k, bias, groups, top)
    assert torch.equal(index.long(), want)
    assert torch.equal(w, weight)


@pytest.mark.parametrize("E,groups,top,k", SOFTMAX)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_a_token_routes_alike_in_every_batch(E, groups, top, k, dtype):
    """Softmax weights and choices of the same rows alone, among more than 2^20 logits (another layout of lanes), and
    where one bias is too large for the fast keys: equal bit for bit."""
    n = 50
    x = (torch.randn(n, E, generator=generator(E + 1), device="cuda") * 1.5).to(KINDS[dtype])
    many = x.repeat((1 << 20) // E // n + 2, 1)
    near = 0.7 - softmax_definition(x[:1], groups)[0]
    for bias in (None, near, near * 0.01) if groups == 1 else (near, near * 0.01):
        how = dict(bias=bias, groups=groups, top_groups=top)
        index, w = route(x, k, **how)
        big_index, big_w = route(many, k, **how)
        assert torch.equal(big_index, index.repeat(many.shape[0] // n, 1))
        assert torch.equal(big_w, w.repeat(many.shape[0] // n, 1))
    close = near.clone()
    close[E - 1] = -2.0 ** 19                                        # never chosen
    far = close.clone()
    far[E - 1] = -2.0 ** 21
    index, w = route(x, k, bias=close, groups=groups, top_groups=top)
    exact_index, exact_w = route(x, k, bias=far, groups=groups, top_groups=top)
    assert torch.equal(exact_index, index) and torch.equal(exact_w, w)

SHAPES = [(1, 1, 1), (5, 8, 2), (33, 32, 8), (7, 33, 4), (300, 60, 4), (40, 64, 6), (65, 128, 8), (20, 200, 12),
          (257, 256, 8), (19, 300, 32), (9, 512, 10), (1201, 16, 3)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k", SHAPES)
def test_gradient_into_contiguous_rows(T, E, k, score, renorm, dtype):
    """Contiguous outputs leave in 16-byte stores where their rows allow it.  Bounds as for strided ones: weights 64u,
    g w summed over k, a score times their sum; rows past the tokens stay as they were."""
    x = (torch.randn(T, E, generator=generator(T), device="cuda") * 1.5).to(KINDS[dtype])
    how = dict(score=score, renorm=renorm, scale=2.5)
    index, w = route(x, k, **how)
    g = torch.randn(T, k, generator=generator(1), device="cuda")
    more = torch.full((T + 2, E), 7.0, dtype=x.dtype, device="cuda")
    d = route_backward(g, x, index, w, out=more[:T], **how)
    assert bool((more[T:] == 7.0).all())
    assert torch.equal(route_backward(g, x, index, w, **how), d)
    wide = torch.full((T, E + 3), 7.0, dtype=x.dtype, device="cuda")
    assert torch.equal(route_backward(g, x, index, w, out=wide[:, :E], **how), d)      # the other path: the same numbers
    got, rows = d.double().cpu().numpy(), x.double().cpu().numpy()
    for t in [*range(min(T, 30)), T - 1]:
        want = R.backward_token(rows[t], index[t].tolist(), g[t].cpu().numpy(), score, renorm, 2.5)
        size = np.abs(g[t].cpu().numpy() * w[t].cpu().numpy()).sum()
        bound = 160 * U * size + (2.0 ** -8 * np.abs(want) if dtype == "bf16" else 0)
        assert np.all(np.abs(got[t] - want) <= bound), t


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("E", [16, 64, 256])
@pytest.mark.parametrize("shift", [1, 2, 3, 5])
def test_logits_that_start_anywhere(E, dtype, shift):
    """Logits, and their gradient, from an address that is no multiple of 16 bytes: what aligned ones give."""
    T, k = 70, 5
    x = (torch.randn(T, E, generator=generator(E), device="cuda") * 1.5).to(KINDS[dtype])
    flat = torch.empty(T * E + 8, dtype=x.dtype, device="cuda")
    odd = flat[shift:shift + T * E].view(T, E)
    odd.copy_(x)
    g = torch.randn(T, k, generator=generator(2), device="cuda")
    out = torch.full((T * E + 8,), 7.0, dtype=x.dtype, device="cuda")
    for score in ("softmax", "sigmoid"):
        for renorm in (False, True):
            how = dict(score=score, renorm=renorm)
            index, w = route(x, k, **how)
            odd_index, odd_w = route(odd, k, **how)
            assert torch.equal(index, odd_index) and torch.equal(w, odd_w)
            d = route_backward(g, x, index, w, **how)
            got = route_backward(g, odd, index, w, out=out[shift:shift + T * E].view(T, E), **how)
            assert torch.equal(got, d)
            assert bool((out[:shift] == 7.0).all()) and bool((out[shift + T * E:] == 7.0).all())
