"""The next-token example's step: its gradients against the same model's in 64 bits and against differences of the loss,
their averages, and the parameters after a step against the oracle's AdamW.

The bound of a gradient: about ten operations one after another, each of sums of at most 16 x 24 terms (fewer than
2^9) with a relative error of at most 2^9 x 2^-24 of its terms' magnitudes, which a layer norm and a softmax pass on; the
terms' magnitudes are taken as at most four times the largest gradient of the tensor: 40 x 2^-15 would be the worst
case, in which all roundings point one way; roundings of either sign add up to the root of that number of terms,
10 x 2^4.5 x 2^-24 x 4 = 5.4e-5, of which twice is allowed."""

import os
import sys

import numpy as np
import pytest
import torch

from oracle import adamw as A
from oracle import tokens as O

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

ROWS, LENGTH = 16, 24


def loss64(params, tokens, targets, seed, X):
    """The example's loss in 64 bits from torch's own operations, with the oracle's dropout."""
    table, w1, b1, matrix, w2, b2 = params

    def factor(x, offset):
        return torch.from_numpy(O.drop(np.ones(tuple(x.shape)), X.P, seed, offset))

    def norm(x, w, b):
        return torch.nn.functional.layer_norm(x, x.shape[-1:], w, b, 1e-5)

    there = (tokens >= 0).unsqueeze(-1)
    x = torch.where(there, table[tokens.clamp(min=0)] * float(np.float32(X.DIM ** 0.5)), torch.zeros((), dtype=torch.float64))
    x = x * factor(x, 0)
    y = torch.tanh(norm(x, w1, b1) @ matrix)
    x = x + y * factor(y, 1)
    logp = torch.log_softmax(norm(x, w2, b2) @ table.t(), -1)
    picked = logp.gather(-1, targets.clamp(min=0).unsqueeze(-1)).squeeze(-1)
    on = targets >= 0
    return -(picked * on).sum() / on.sum()


def test_a_step_equals_the_formula():
    import token_training_step as X
    gen = torch.Generator("cuda").manual_seed(5)
    model = X.Model(gen)
    trainer = X.Trainer(model, replicas=2)
    w = [p.detach().cpu().double() for p in model.params]
    m, v = ([np.zeros(p.numel()) for p in w] for _ in range(2))
    for t in (1, 2):
        batch = X.batches(2, ROWS, LENGTH, gen)
        loss = float(trainer.step(batch))
        torch.cuda.synchronize()
        losses = []
        for r, (tokens, targets) in enumerate(batch):
            leaves = [p.clone().requires_grad_(True) for p in w]
            want = loss64(leaves, tokens.cpu(), targets.cpu(), t * 2 + r, X)
            losses.append(float(want.detach()))
            for g, d in zip(trainer.fields[r], torch.autograd.grad(want, leaves)):
                assert float((g.cpu().double() - d).abs().max()) <= 1.1e-4 * float(d.abs().max())
        assert loss == pytest.approx(np.mean(losses), rel=1e-5)
        mean = [(a.double() + b.double()).cpu().numpy() / 2 for a, b in zip(*trainer.grads)]
        for g, d in zip(trainer.mean, mean):
            np.testing.assert_allclose(g.cpu().numpy(), d, rtol=2.0 ** -22, atol=2.0 ** -24 * np.abs(d).max())
        norm = A.grad_norm(mean)
        assert float(trainer.norm) == pytest.approx(norm, rel=1e-6)
        clip = A.clip_factor(norm, 1.0)
        for i, p in enumerate(model.params):
            wd = 0.01 if p.dim() > 1 else 0.0
            after, m[i], v[i] = A.adamw(w[i].numpy().reshape(-1), mean[i], m[i], v[i], t, 3e-3, 0.9, 0.999, 1e-8, wd, clip)
            now = p.detach().cpu().double()
            # fp32 roundings of w, and a relative 1e-4 of a step where a gradient is so small that eps tells
            np.testing.assert_allclose(now.numpy().reshape(-1), after, rtol=0,
                                       atol=2.0 ** -23 * np.abs(after).max() + 3 * 3e-3 * 1e-4)
            w[i] = now                                             # the next step begins with what this one left


def test_gradients_equal_differences():
    """Along the gradient g of every parameter: the loss changes by eps |g|^2 x (1 + O(eps^2)), and the losses' own
    roundings, about 2^-20 of 5, come to 5e-6 / (2 eps |g|) of that; eps |g| = 1/50 leaves well under 1 %."""
    import token_training_step as X
    gen = torch.Generator("cuda").manual_seed(6)
    model = X.Model(gen)
    trainer = X.Trainer(model, replicas=1)
    (tokens, targets), = X.batches(1, ROWS, LENGTH, gen)
    trainer.backward(0, tokens, targets)
    field = [g.clone() for g in trainer.fields[0]]
    for p, g in zip(model.params, field):
        size = float(g.norm())
        eps, at = 0.02 / size, []
        for sign in (1, -1):
            with torch.no_grad():
                p.add_(g, alpha=sign * eps)
                at.append(float(model.loss(tokens, targets, 0, trainer.fields[0])))
                p.sub_(g, alpha=sign * eps)
        assert (at[0] - at[1]) / (2 * eps * size) == pytest.approx(size, rel=0.02)


def test_it_runs():
    import token_training_step as X
    losses = X.main(steps=3)
    assert len(losses) == 3 and np.isfinite(losses).all()
