"""The example's training step, run through the library and by hand: gradients averaged and clipped in 64 bits from the
same replicas' gradients, the oracle's AdamW on the parameters that were used, the others untouched."""

import os
import sys

import numpy as np
import pytest
import torch

from oracle import adamw as A

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def test_steps_equal_the_formula():
    import expert_training_step as X
    gen = torch.Generator("cuda").manual_seed(3)
    model = X.Experts(gen)
    trainer = X.Trainer(model, replicas=2, state_bits=32)
    teacher = torch.randn(X.DIM, X.DIM, generator=gen, device="cuda") / X.DIM ** 0.5
    w = [p.detach().cpu().numpy().reshape(-1).astype(np.float64) for p in model.params]
    m, v = [np.zeros_like(x) for x in w], [np.zeros_like(x) for x in w]
    unused = 0
    for t in range(1, 6):
        before = [p.detach().clone() for p in model.params]
        trainer.step(X.batches(teacher, 2, 6, gen))       # few tokens: some experts get none
        torch.cuda.synchronize()
        mean = []
        for i in range(len(w)):
            parts = [trainer.grads[r][i].cpu().numpy().astype(np.float64) if trainer.local[r][i] else np.zeros(w[i].size)
                     for r in range(2)]
            mean.append((parts[0] + parts[1]) / 2)
        norm = A.grad_norm([g for g, u in zip(mean, trainer.used) if u])
        assert float(trainer.norm) == pytest.approx(norm, rel=1e-6)
        clip = A.clip_factor(norm, 1.0)
        for i, p in enumerate(model.params):
            now = p.detach().cpu().numpy().reshape(-1).astype(np.float64)
            if not trainer.used[i]:
                unused += 1
                assert torch.equal(p.detach(), before[i])
                continue
            wd = 0.01 if p.dim() > 1 else 0.0
            w[i], m[i], v[i] = A.adamw(w[i], mean[i], m[i], v[i], t, 3e-3, 0.9, 0.999, 1e-8, wd, clip)
            # a step is at most about lr x 3; fp32 roundings of w over five steps, and a relative 1e-5 of the update
            # where a gradient is so small that eps tells
            np.testing.assert_allclose(now, w[i], rtol=0, atol=5 * 2 ** -23 * np.abs(w[i]).max() + 5 * 3e-3 * 1e-4)
            w[i] = now
    assert unused > 0


@pytest.mark.parametrize("bits", [32, 8])
def test_the_loss_falls(bits):
    import expert_training_step as X
    losses = X.main(steps=150, state_bits=bits)
    assert np.mean(losses[-10:]) < 0.6 * np.mean(losses[:5])
