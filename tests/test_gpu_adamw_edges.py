"""Edges of the AdamW step and the gradient norm on the GPU: the default rounding, moments near fp32's least numbers and
beside its largest, calls on another stream after a bind, one optimizer bound again and again."""

import numpy as np
import pytest
import torch

from reduction_reducer_gb300 import AdamW

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _device():
    torch.cuda.set_device(0)

def test_steps_without_a_seed_round_anew_each_time():
    """step(t) alone, 3000 times: with the same random bits in every step an element's rounding threshold never moves,
    and its second moment stays where that holds it.  The mean over 65,536 elements (noise of the rounding 30 % an
    element, 0.12 % in the mean) lies within 2 % of the 32-bit run's, from a start four times too high."""
    n, sigma = 65536, 1e-2
    gen = torch.Generator("cuda").manual_seed(1)
    runs = {}
    for bits in (32, 8):
        opt = AdamW([n], "f32", bits)
        w, g = torch.zeros(n, device="cuda"), torch.empty(n, device="cuda")
        state = opt.zero_state()
        if bits == 32:
            state["exp_avg_sq"][0].fill_(4 * sigma ** 2)
        else:
            state["exp_avg_sq"][0].copy_(torch.ones(n, device="cuda").to(torch.float8_e5m2))
            state["exp_avg_sq_scale"][0].fill_(4 * sigma ** 2)
        opt.bind([w], [g], **state)
        gen.manual_seed(2)
        for t in range(1, 3001):
            g.normal_(generator=gen).mul_(sigma)
            opt.step(t)
        x = state["exp_avg_sq"][0].float()
        if bits == 8:
            x = x * state["exp_avg_sq_scale"][0].repeat_interleave(256)
        runs[bits] = float(x.mean())
    assert abs(runs[8] / runs[32] - 1) < 0.02


def test_the_default_seed_is_the_step():
    g = torch.randn(5000, generator=torch.Generator("cuda").manual_seed(0), device="cuda")
    made = []
    for seeds in ({}, dict(seed=7), dict(seed=8), dict(seed=0)):
        opt = AdamW([5000], "f32", 8)
        w, state = torch.zeros(5000, device="cuda"), opt.zero_state()
        opt.bind([w], [g], **state)
        opt.step(7, **seeds)
        made.append(state["exp_avg"][0].view(torch.uint8).clone())
    assert torch.equal(made[0], made[1])
    assert not torch.equal(made[0], made[2]) and not torch.equal(made[0], made[3])

@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_second_moments_below_the_least_normal_number(dtype, bits):
    """The first step from zero state moves a weight by lr, however small the gradient: g of 3e-19 to 3e-18 gives v of
    9e-41 to 9e-39, below 2^-126, whose rounding (2^-150 of it, half of that of its root) is at most 4e-6."""
    n = 1000
    gen = torch.Generator("cuda").manual_seed(0)
    sign = torch.where(torch.rand(n, generator=gen, device="cuda") < 0.5, -1.0, 1.0)
    g = sign * 3e-19 * 10 ** torch.rand(n, generator=gen, device="cuda")
    opt = AdamW([n], dtype, bits)
    w = torch.zeros(n, device="cuda")
    bf16 = dict(master=[w]) if dtype == "bf16" else {}
    opt.bind([w.bfloat16() if bf16 else w], [g], **bf16, **opt.zero_state())
    opt.step(1, lr=0.5, eps=1e-30)
    v = 1e-3 * g.double() ** 2
    assert float(v.max()) < 2.0 ** -126
    assert bool(((w.double() + 0.5 * sign).abs() <= 0.5 * (24 * U + 2.0 ** -151 / v)).all())


@pytest.mark.parametrize("bits", [32, 8])
def test_second_moments_near_the_largest_number(bits):
    """g of 1e13 to 1e19, v of 1e23 to 1e35, beside small ones in the same blocks: each first step moves its weight by lr."""
    n = 1000
    g = torch.logspace(13, 19, n, device="cuda")
    g[1::2] = 10.0 ** -torch.linspace(0, 5, n // 2, device="cuda")
    opt = AdamW([n], "f32", bits)
    w = torch.zeros(n, device="cuda")
    opt.bind([w], [g], **opt.zero_state())
    opt.step(1, lr=0.5, eps=1e-30)
    assert bool(((w + 0.5).abs() <= 0.5 * 24 * U).all())

@pytest.mark.parametrize("size", [1e-16, 1e-17, 1e-18])
def test_eight_bit_moments_of_tiny_gradients(size):
    """Blocks whose largest second moment over 57344 is no normal number keep their moments too.  m is within an eighth
    of itself and v within a quarter, or half a spacing, of the unrounded ones; a step of equal gradients moves a weight
    by lr to within the errors of both, and one without a gradient by less."""
    n, steps = 600, 8
    opt = AdamW([n], "f32", 8)
    w, g = torch.zeros(n, device="cuda"), torch.full((n,), size, device="cuda")
    state = opt.zero_state()
    opt.bind([w], [g], **state)
    for t in range(1, steps + 1):
        opt.step(t, lr=0.5, eps=1e-30, seed=t)
    assert bool((state["exp_avg_sq"][0].float() > 0).all())
    m = state["exp_avg"][0].float() * state["exp_avg_scale"][0].repeat_interleave(256)[:n]
    v = state["exp_avg_sq"][0].double() * state["exp_avg_sq_scale"][0].double().repeat_interleave(256)[:n]
    assert float(m.mean()) == pytest.approx(size * (1 - 0.9 ** steps), rel=0.02)
    assert float(v.mean()) == pytest.approx(size ** 2 * (1 - 0.999 ** steps), rel=0.05)
    assert float((w / (-0.5 * steps)).mean()) == pytest.approx(1.0, rel=0.05)
    before = w.clone()
    g.zero_()
    opt.step(steps + 1, lr=0.5, eps=1e-30, seed=steps + 1)
    assert float((w - before).abs().max()) <= 0.5 * 1.5

def test_a_second_moment_beside_a_huge_one_is_not_stored_as_zero():
    """v of 1e-15 in a block whose largest is 2e35: their quotient by the scale is below fp32's least number."""
    n = 256
    opt = AdamW([n], "f32", 8)
    w, g = torch.zeros(n, device="cuda"), torch.full((n,), 1e-6, device="cuda")
    g[0] = 1.5e19
    state = opt.zero_state()
    opt.bind([w], [g], **state)
    opt.step(1, seed=1)
    scale = float(state["exp_avg_sq_scale"][0][0])
    assert np.isfinite(scale) and np.float32(1e-15) / np.float32(scale) == 0
    assert bool((state["exp_avg_sq"][0].float() > 0).all())

def test_steps_on_another_stream_follow_each_bind():
    """Each bind's table is the one that calls on a stream of their own then read: gradients and weights alternate, so a
    table of the bind before would show in the norm and in the weights."""
    sizes = [1 + v % 5 for v in range(900)]
    total = sum(sizes)
    opt = AdamW(sizes)
    state = opt.zero_state()
    side = torch.cuda.Stream()
    norm = torch.zeros(1, device="cuda")
    sets = []
    for x in (2.0, -3.0):
        sets.append((x, [torch.full((n,), x, device="cuda") for n in sizes], [torch.zeros(n, device="cuda") for n in sizes]))
    torch.cuda.synchronize()
    for i in range(12):
        x, g, w = sets[i % 2]
        for views in state.values():
            for s in views:
                s.zero_()
        for t in w:
            t.zero_()
        norm.zero_()
        torch.cuda.synchronize()
        opt.bind(w, g, **state)
        opt.grad_norm(norm, stream=side)
        opt.step(1, lr=0.25, stream=side)
        side.synchronize()
        assert float(norm) == pytest.approx(abs(x) * total ** 0.5, rel=1e-6)
        assert torch.allclose(torch.cat(w), torch.full((total,), -0.25 if x > 0 else 0.25, device="cuda"), rtol=24 * U, atol=0)
        other = torch.cat(sets[1 - i % 2][2])
        assert i == 0 or bool((other.abs() > 0).all())               # the set before stays as its own step left it
        torch.cuda.synchronize()


def test_one_optimizer_bound_again_and_again():
    """Norms before and after binds of one optimizer to other tensors, with and without parameters; of grids that change
    with the tensors that are left out."""
    sizes = [700_000, 5, 1_500_000]
    total = sum(sizes)
    opt = AdamW(sizes)
    norm = torch.zeros(1, device="cuda")
    used = torch.tensor([1, 1, 0], dtype=torch.uint8, device="cuda")
    for x in (0.5, 2.0, 0.25, 3.0):
        g = [torch.full((n,), x, device="cuda") for n in sizes]
        if x > 1:
            opt.bind_grads(g)
        else:
            opt.bind([torch.zeros_like(t) for t in g], g, **opt.zero_state())
        for _ in range(3):
            assert float(opt.grad_norm(norm)) == pytest.approx(x * total ** 0.5, rel=1e-6)
            assert float(opt.grad_norm(norm, used=used)) == pytest.approx(x * 700_005 ** 0.5, rel=1e-6)
