"""Training steps of a small mixture of experts on W data-parallel replicas of one GPU.

Each step runs what this package has around a backward pass, in order:

* ``routed``: tokens to experts, with the number of tokens each expert got;
* these counts are the local-use bits of the experts' parameters: an expert
  that no token of a replica reached has no gradient there
  (``Reducer.set_local_used``), one that no token reached at all keeps its
  parameters and moments;
* ``Reducer``: the replicas' gradients, averaged bucket by bucket into the
  arena, whose views are the gradients from there on;
* ``AdamW.grad_norm`` and ``AdamW.step`` on these views, with 8-bit moments;
* the balance bias moves towards the experts that got too few tokens.

    python examples/expert_training_step.py [steps]
"""

from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from reduction_reducer_gb300 import AdamW, Reducer, _lib, routed  # noqa: E402

DIM, HIDDEN, EXPERTS, K, GROUPS, TOP_GROUPS = 32, 48, 16, 2, 4, 2


class Experts:
    """A linear router and EXPERTS two-layer networks, as a list of parameters in registration order."""

    def __init__(self, generator):
        def normal(*shape):
            return torch.randn(*shape, generator=generator, device="cuda") / shape[0] ** 0.5

        self.router = normal(DIM, EXPERTS)
        self.experts = [(normal(DIM, HIDDEN), torch.zeros(HIDDEN, device="cuda"), normal(HIDDEN, DIM) * 0.1)
                        for _ in range(EXPERTS)]
        self.bias = torch.zeros(EXPERTS, device="cuda")                  # of the choice; not learned by gradient
        self.params = [self.router] + [p for e in self.experts for p in e]
        self.owner = [None] + [e for e in range(EXPERTS) for _ in range(3)]   # the expert of each parameter
        for p in self.params:
            p.requires_grad_(True)

    def __call__(self, x, counts):
        index, weight = routed(x @ self.router, K, score="sigmoid", bias=self.bias, groups=GROUPS,
                               top_groups=TOP_GROUPS, renorm=True, counts=counts)
        out = torch.zeros_like(x)
        for e, (w1, b1, w2) in enumerate(self.experts):
            token, slot = (index == e).nonzero(as_tuple=True)
            if len(token):
                h = torch.relu(x[token] @ w1 + b1) @ w2
                out = out.index_add(0, token, h * weight[token, slot].unsqueeze(1))
        return out


class Trainer:
    def __init__(self, model, replicas, state_bits=8, lr=3e-3, max_norm=1.0):
        self.model, self.W, self.lr, self.max_norm, self.t = model, replicas, lr, max_norm, 0
        numel = [p.numel() for p in model.params]
        self.grads = [[torch.zeros(n, device="cuda") for n in numel] for _ in range(replicas)]
        self.reducer = Reducer(numel, "f32", 16 << 10)
        self.reducer.set_option(_lib.OPT_FIND_UNUSED, 1)
        self.arena = torch.zeros(self.reducer.arena_numel(), device="cuda")
        self.reducer.bind(self.grads, self.arena, None)                  # the gradients are bucket views
        _, offsets = self.reducer.get_bucket_info()
        self.mean = [self.arena[offsets[b] + o:offsets[b] + o + n] for b, _, o, n in self.reducer.get_locators()]
        self.opt = AdamW(numel, state_bits=state_bits)
        self.state = self.opt.zero_state()
        self.opt.bind([p.detach().view(-1) for p in model.params], self.mean,
                      weight_decay=[0.01 if p.dim() > 1 else 0.0 for p in model.params], **self.state)
        self.norm = torch.zeros(1, device="cuda")

    def step(self, batches):
        """One step on one (input, target) batch per replica; the mean loss."""
        model, self.t, losses = self.model, self.t + 1, []
        counts = torch.zeros(self.W, EXPERTS, dtype=torch.int32, device="cuda")
        for r, (x, y) in enumerate(batches):
            loss = (model(x, counts[r]) - y).square().mean()
            for buffer, g in zip(self.grads[r], torch.autograd.grad(loss, model.params, allow_unused=True)):
                if g is not None:
                    buffer.copy_(g.reshape(-1))
            losses.append(loss.detach())
        got = (counts > 0).cpu().tolist()
        self.local = [[e is None or got[r][e] for e in model.owner] for r in range(self.W)]
        self.used = [any(bits) for bits in zip(*self.local)]
        self.reducer.set_local_used(self.local)
        self.reducer.begin_iteration()
        for v in reversed(range(len(model.params))):                     # as a backward pass reports them
            if self.used[v]:
                self.reducer.mark_ready(v)
        used = torch.tensor(self.used, device="cuda")
        self.opt.grad_norm(self.norm, used=used)
        self.opt.step(self.t, lr=self.lr, norm=self.norm, max_norm=self.max_norm, used=used, seed=self.t,
                      skip_nonfinite=True)
        total = counts.sum(0)
        model.bias += 1e-3 * torch.sign(total.float().mean() - total)
        return torch.stack(losses).mean()


def batches(teacher, replicas, tokens, generator):
    x = [torch.randn(tokens, DIM, generator=generator, device="cuda") for _ in range(replicas)]
    return [(b, torch.tanh(b @ teacher)) for b in x]


def main(steps=200, replicas=2, tokens=256, state_bits=8):
    generator = torch.Generator("cuda").manual_seed(0)
    trainer = Trainer(Experts(generator), replicas, state_bits)
    teacher = torch.randn(DIM, DIM, generator=generator, device="cuda") / DIM ** 0.5
    losses = []
    for t in range(steps):
        losses.append(float(trainer.step(batches(teacher, replicas, tokens, generator))))
        if t % 20 == 0 or t + 1 == steps:
            print(f"step {t + 1:4d}  loss {losses[-1]:.4f}  norm {float(trainer.norm):.3f}  "
                  f"tensors with a gradient {sum(trainer.used)} of {len(trainer.used)}")
    return losses


if __name__ == "__main__":
    main(int(sys.argv[1]) if len(sys.argv) > 1 else 200)
