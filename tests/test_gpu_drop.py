"""Dropout on the GPU against the 64-bit oracle: which elements stay is whole numbers, and has to be equal; a value is
x times an fp32 scale (u each: 2 u) plus the residual (u), rounded once more (h)."""

import numpy as np
import pytest
import torch

from oracle import tokens as O
from reduction_reducer_gb300 import drop, dropped

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
KINDS = {"f32": torch.float32, "bf16": torch.bfloat16}
HALF = {"f32": U, "bf16": 2.0 ** -8}


@pytest.fixture(scope="module", autouse=True)
def _device():
    torch.cuda.set_device(0)


def rows(n, dim, kind, seed, extra=0, shift=0):
    gen = torch.Generator("cuda").manual_seed(seed)
    flat = torch.randn(n * (dim + extra) + shift, generator=gen, device="cuda").to(KINDS[kind])
    return flat[shift:].as_strided((n, dim), (dim + extra, 1))


def host(t):
    return t.double().cpu().numpy()


def check(got, x, p, seed, offset, residual, kind):
    want = O.drop(host(x), p, seed, offset, None if residual is None else host(residual))
    kept = np.abs(O.drop(host(x), p, seed, offset))
    bound = 3 * U * kept + (U + HALF[kind] * (1 + 2 ** -6)) * np.abs(want)
    assert np.all(np.abs(host(got) - want) <= bound)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("n,dim", [(1, 1), (1, 7), (3, 8), (5, 24), (7, 33), (2, 1029), (40, 64)])
def test_drop(n, dim, kind):
    for p, seed, offset in ((0.1, 0, 0), (0.5, 2 ** 64 - 1, 2 ** 63 - 1), (0.37, 12345678901234567, 5)):
        for extra, shift in ((0, 0), (8, 0), (3, 1)):
            x, r = rows(n, dim, kind, 1, extra, shift), rows(n, dim, kind, 2, extra, shift)
            for residual in (None, r):
                wide = torch.full((n, dim + 8), 7.0, dtype=x.dtype, device="cuda")
                got = drop(x, p, seed, offset, residual, out=wide[:, :dim])
                check(got, x, p, seed, offset, residual, kind)
                assert bool((wide[:, dim:] == 7.0).all())
                # the same elements whatever the layout
                assert torch.equal(drop(x.contiguous(), p, seed, offset, residual), got)


def test_the_border_counts_in_32_bits():
    """Probabilities whose upper half is an element's own: the lower half decides."""
    n, seed, offset = 64, 77, 9
    x = torch.ones(1, n, device="cuda")
    bits = [O.random_bits(e, seed, offset) for e in range(n)]
    for e in (0, 1, 6, 7, 8, 63):
        for p, stays in ((bits[e] / 2 ** 32, True), ((bits[e] + 1) / 2 ** 32, False)):
            y = drop(x, p, seed, offset)
            assert bool(y[0, e] != 0) == stays
            assert [bool(v) for v in (y[0] != 0).tolist()] == [b >= round(p * 2 ** 32) for b in bits]


def test_all_and_none():
    x = torch.tensor([[1.0, float("nan"), float("inf"), -0.0, 5.0]], device="cuda")
    assert torch.equal(drop(x, 1.0, 3), torch.zeros_like(x))
    assert torch.equal(drop(x, 1 - 2.0 ** -40, 3), torch.zeros_like(x))
    assert torch.equal(drop(x, 0.0, 3)[0, [0, 2, 3, 4]], x[0, [0, 2, 3, 4]])
    assert torch.equal(drop(x, 1.0, 3, residual=torch.ones_like(x)), torch.ones_like(x))
    assert drop(torch.empty(0, 5, device="cuda"), 0.5, 1).shape == (0, 5)
    assert drop(torch.empty(5, 0, device="cuda"), 0.5, 1).shape == (5, 0)


def test_in_place_and_device_seed():
    x, r = rows(9, 100, "bf16", 1), rows(9, 100, "bf16", 2)
    want = drop(x, 0.3, 5, 1, r)
    a, b = x.clone(), r.clone()
    assert torch.equal(drop(a, 0.3, 5, 1, r, out=a), want) and torch.equal(a, want)
    assert torch.equal(drop(x, 0.3, 5, 1, b, out=b), want)
    seed = torch.tensor([5], device="cuda")
    assert torch.equal(drop(x, 0.3, seed, 1, r), want)
    # a captured call draws anew where its seed is on the device
    graph, out = torch.cuda.CUDAGraph(), torch.empty_like(x)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        drop(x, 0.3, seed, 1, r, out=out)
    for s in (5, 2 ** 62 + 3, -1):
        seed.fill_(s)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, drop(x, 0.3, s % 2 ** 64, 1, r))


def test_rates_and_independence():
    """Of n elements the share that stays is within five standard deviations; neighbours, seeds and offsets agree as
    chance has it."""
    n, p = 1 << 22, 0.3
    x = torch.ones(n, device="cuda")
    masks = [drop(x, p, s, o) != 0 for s, o in ((1, 0), (2, 0), (1, 1), (1 << 32, 0), (1, 1 << 32))]
    for m in masks:
        assert abs(m.double().mean().item() - 0.7) < 5 * (0.21 / n) ** 0.5
        both = (m[1:] & m[:-1]).double().mean().item()
        assert abs(both - 0.49) < 5 * (0.25 * 2 / n) ** 0.5
    for i in range(len(masks)):
        for j in range(i):
            assert abs((masks[i] & masks[j]).double().mean().item() - 0.49) < 5 * (0.25 / n) ** 0.5


def test_autograd():
    x, r = (rows(6, 50, "f32", s).contiguous().requires_grad_(True) for s in (1, 2))
    y = dropped(x, 0.4, 11, 3, r)
    assert torch.equal(y, drop(x.detach(), 0.4, 11, 3, r.detach()))
    g = rows(6, 50, "f32", 3)
    y.backward(g)
    assert torch.equal(x.grad, drop(g, 0.4, 11, 3)) and torch.equal(r.grad, g)
    x.grad = None
    dropped(x, 0.4, 11, 3).sum().backward()
    assert torch.equal(x.grad, drop(torch.ones_like(g), 0.4, 11, 3))
    x.grad = None
    dropped(x.view(2, 3, 50).transpose(0, 1).contiguous(), 0.4, 11, 3).mean().backward()
    assert x.grad.count_nonzero() > 0
