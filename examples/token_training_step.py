"""Training steps of a small next-token model on W data-parallel replicas of one GPU.

Each step runs what this package has around the matrix products, in order:

* ``embedded`` and ``dropped``: tokens to rows, some of their elements dropped;
* ``layer_normed``, a product, ``dropped`` onto the residual, ``layer_normed``;
* a product with the embedding's table, and ``scored``: the targets' log
  probabilities; those of padding are left out;
* the backward pass: the norms' and the embedding's gradients go into the
  replica's gradient fields at once (``grad_into``), and the product's with the
  table is added to the embedding's;
* ``Reducer``: the replicas' gradients, averaged bucket by bucket into the
  arena, whose views are the gradients from there on;
* ``AdamW.grad_norm`` and ``AdamW.step`` on these views.

    python examples/token_training_step.py [steps]
"""

from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from reduction_reducer_gb300 import AdamW, Reducer, dropped, embedded, layer_normed, scored  # noqa: E402

VOCAB, DIM, P = 61, 40, 0.1


class Model:
    """A table, two layer norms and a matrix, as a list of parameters in registration order."""

    def __init__(self, generator):
        def normal(*shape):
            return torch.randn(*shape, generator=generator, device="cuda")

        self.params = [normal(VOCAB, DIM) * 0.3, 1 + 0.1 * normal(DIM), 0.1 * normal(DIM), normal(DIM, DIM) / DIM ** 0.5,
                       1 + 0.1 * normal(DIM), 0.1 * normal(DIM)]
        for p in self.params:
            p.requires_grad_(True)

    def loss(self, tokens, targets, seed, into):
        """The targets' mean negative log probability.  into: a gradient field for each parameter, [its shape]."""
        table, w1, b1, matrix, w2, b2 = self.params
        x = dropped(embedded(table, tokens, scale=DIM ** 0.5, grad_into=into[0]), P, seed, offset=0)
        y = torch.tanh(layer_normed(x, w1, b1, grad_into=(into[1], into[2])) @ matrix)
        x = dropped(y, P, seed, offset=1, residual=x)
        y = layer_normed(x, w2, b2, grad_into=(into[4], into[5]))
        logp = scored(y @ table.t(), targets).logp              # 0 where there is no target
        return -logp.sum() / ((targets >= 0) & (targets < VOCAB)).sum()


class Trainer:
    def __init__(self, model, replicas, lr=3e-3, max_norm=1.0):
        self.model, self.W, self.lr, self.max_norm, self.t = model, replicas, lr, max_norm, 0
        numel = [p.numel() for p in model.params]
        self.grads = [[torch.zeros(n, device="cuda") for n in numel] for _ in range(replicas)]
        self.fields = [[g.view(p.shape) for g, p in zip(grads, model.params)] for grads in self.grads]
        self.reducer = Reducer(numel, "f32", 16 << 10)
        self.arena = torch.zeros(self.reducer.arena_numel(), device="cuda")
        self.reducer.bind(self.grads, self.arena, None)                  # the gradients are bucket views
        _, offsets = self.reducer.get_bucket_info()
        self.mean = [self.arena[offsets[b] + o:offsets[b] + o + n] for b, _, o, n in self.reducer.get_locators()]
        self.opt = AdamW(numel)
        self.opt.bind([p.detach().view(-1) for p in model.params], self.mean,
                      weight_decay=[0.01 if p.dim() > 1 else 0.0 for p in model.params], **self.opt.zero_state())
        self.norm = torch.zeros(1, device="cuda")

    def backward(self, r, tokens, targets):
        """Replica r's gradients into its fields; the loss."""
        for field in self.fields[r]:
            field.zero_()
        loss = self.model.loss(tokens, targets, self.t * self.W + r, self.fields[r])
        for field, g in zip(self.fields[r], torch.autograd.grad(loss, self.model.params, allow_unused=True)):
            if g is not None:                                            # of the two products
                field += g
        return loss.detach()

    def step(self, batches):
        """One step on one (tokens, targets) batch per replica; the mean loss."""
        self.t += 1
        losses = [self.backward(r, *batch) for r, batch in enumerate(batches)]
        self.reducer.begin_iteration()
        for v in reversed(range(len(self.model.params))):                # as a backward pass reports them
            self.reducer.mark_ready(v)
        self.opt.grad_norm(self.norm)
        self.opt.step(self.t, lr=self.lr, norm=self.norm, max_norm=self.max_norm, seed=self.t, skip_nonfinite=True)
        return torch.stack(losses).mean()


def batches(replicas, rows, length, generator):
    """Sequences in which each token decides on the next one, of several lengths: -1 behind their ends."""
    out = []
    for _ in range(replicas):
        tokens = torch.randint(VOCAB, (rows, 1), generator=generator, device="cuda")
        for _ in range(length):
            tokens = torch.cat([tokens, (tokens[:, -1:] * 5 + 3) % VOCAB], 1)
        ends = torch.randint(1, length + 1, (rows, 1), generator=generator, device="cuda")
        behind = torch.arange(length, device="cuda") >= ends
        out.append((tokens[:, :-1].masked_fill(behind, -1), tokens[:, 1:].masked_fill(behind, -1)))
    return out


def main(steps=200, replicas=2, rows=16, length=24):
    generator = torch.Generator("cuda").manual_seed(0)
    trainer = Trainer(Model(generator), replicas)
    losses = []
    for t in range(steps):
        losses.append(float(trainer.step(batches(replicas, rows, length, generator))))
        if t % 20 == 0 or t + 1 == steps:
            print(f"step {t + 1:4d}  loss {losses[-1]:.4f}  norm {float(trainer.norm):.3f}")
    return losses


if __name__ == "__main__":
    main(int(sys.argv[1]) if len(sys.argv) > 1 else 200)
