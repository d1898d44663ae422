"""Log probabilities, entropy, alternatives and the logits' gradient on the GPU against the 64-bit oracle.

Bounds (u = 2^-24; d = z - m).  An exponential errs by 4 u (its approximation) and 3 u |d| (difference, scale and
base), at most 3 u 0.4 of the largest term.  A sum has 32 terms of a batch, up to B = 16 batches of a thread (7 u each,
with the rescaling of the earlier ones) and 12 steps of joining (8 u each): 250 u with the exponential's; so log S errs
by 250 u + 2 u log S, and the mean of d by twice that of itself.  log p: 4 u |d| and log S's; the entropy the sum of both
and 2 u.  A gradient, from statistics rounded to fp32: log p = z - M - L with M = m (1 + e), L = log S (1 + e'), |e| and
|e'| at most u, is off by (|m| + log S) u and, with its own roundings, 4 u |log p|; p by that and 8 u of itself; the
factor g + h (log p + H) by 8 u of its terms and by |h| times what log p and H (rounded: u H) are off by."""

import numpy as np
import pytest
import torch

from oracle import tokens as O
from reduction_reducer_gb300 import logprobs, logprobs_backward, scored

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
KINDS = {"f32": torch.float32, "bf16": torch.bfloat16}
HALF = {"f32": U, "bf16": 2.0 ** -8}
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module", autouse=True)
def _device():
    torch.cuda.set_device(0)


def generator(seed):
    return torch.Generator("cuda").manual_seed(seed)


def draw(n, vocab, kind, seed, extra=0, shift=0, spread=2.0):
    flat = torch.randn(n * (vocab + extra) + shift, generator=generator(seed), device="cuda") * spread
    return flat.to(KINDS[kind])[shift:].as_strided((n, vocab), (vocab + extra, 1))


def draw_targets(n, vocab, seed, masked=True):
    t = torch.randint(vocab, (n,), generator=generator(seed), device="cuda")
    if masked and n > 2:
        t[1], t[-1] = -100, vocab
    return t


def host(t):
    return None if t is None else t.detach().double().cpu().numpy()


def near(got, want, bound):
    """Within the bound where finite, and of the same kind elsewhere."""
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    fine = np.isfinite(want)
    return np.array_equal(got[~fine], want[~fine], equal_nan=True) and np.all(
        np.abs(got[fine] - want[fine]) <= np.broadcast_to(bound, got.shape)[fine])


def check(x, targets, top, scale, got, entropy=True):
    t = None if targets is None else targets.cpu().tolist()
    rows, s32 = host(x), float(np.float32(scale))
    logp, ent, stats, index, top_logp = (host(v) for v in got)
    assert (ent is None) == (not entropy) and (logp is None) == (targets is None)
    for i in range(len(rows)):
        want, h, (m, log_s), order, alternatives = O.logprobs(rows[i], None if t is None else t[i], top, s32)
        slack = 250 * U + 2 * U * abs(log_s) if np.isfinite(log_s) else 0
        spent = abs(h - log_s) if np.isfinite(h) else 0          # |mean of d|
        assert near(stats[i], (m, log_s), (U * abs(m) if np.isfinite(m) else 0, slack))
        if t is not None:
            assert near(logp[i], want, slack + 4 * U * abs(want) + 4 * U * abs(want + log_s))
        if entropy:
            assert near(ent[i], h, slack + 500 * U * spent + 3 * U * abs(h))
        if top:
            assert index[i].astype(int).tolist() == order, (i, index[i], order)
            a = np.array(alternatives)
            assert near(top_logp[i], a, slack + 8 * U * np.where(np.isfinite(a), np.abs(a) + abs(log_s), 0))


SHAPES = [(1, 1), (3, 2), (9, 7), (5, 100), (17, 256), (4, 1000), (3, 2047), (3, 2048), (3, 2049), (5, 5003), (3, 16384),
          (4, 30522), (5, 50257), (2, 131072)]


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("n,vocab", SHAPES)
def test_forward(n, vocab, kind):
    for extra, shift, scale, bits in ((0, 0, 1.0, torch.int64), (3, 1, 0.7, torch.int32), (8, 0, 1.3, torch.int64)):
        x, t = draw(n, vocab, kind, vocab, extra, shift), draw_targets(n, vocab, 1).to(bits)
        top = min(vocab, 8 if extra else 32)
        full = logprobs(x, t, top, scale, entropy=True)
        check(x, t, top, scale, full)
        bare = logprobs(x, t, 0, scale)
        check(x, t, 0, scale, bare, entropy=False)
        # what is asked for does not change the rest
        assert torch.equal(bare.logp, full.logp) and torch.equal(bare.stats, full.stats)
        assert torch.equal(logprobs(x, t, 0, scale, entropy=True).entropy, full.entropy)
        check(x, None, 1, scale, logprobs(x, None, 1, scale), entropy=False)


@pytest.mark.parametrize("n", [1, 40, 400])
def test_a_row_is_the_same_alone(n):
    """Rows split over CTAs and rows that are not differ in the order of sums alone; alternatives are equal."""
    x, t = draw(n, 50257, "bf16", 3), draw_targets(n, 50257, 4, masked=False)
    many, one = logprobs(x, t, 10, entropy=True), logprobs(x[:1], t[:1], 10, entropy=True)
    assert torch.equal(many.top_index[:1], one.top_index)
    assert torch.allclose(many.logp[:1], one.logp, rtol=0, atol=500 * U)
    assert torch.allclose(many.entropy[:1], one.entropy, rtol=0, atol=1000 * U)


@pytest.mark.parametrize("vocab", [40, 2048, 3001, 50257])
def test_ties_go_to_the_lowest(vocab):
    for kind in KINDS:
        x = torch.zeros(4, vocab, dtype=KINDS[kind], device="cuda")
        x[1] = -0.0
        x[1, 5::2] = 0.0
        x[2] = torch.arange(vocab, device="cuda").flip(0) // 7                # descending, in sevens
        x[3] = torch.arange(vocab, device="cuda") // 7                        # ascending
        for top in (1, 20, 32):
            got = logprobs(x, None, top, entropy=True)
            check(x, None, top, 1.0, got)
            assert got.top_index[0].tolist() == list(range(top)) == got.top_index[1].tolist()


def test_many_ties_and_many_large_in_one_thread():
    """A thread of a row that holds many of the largest, and coarse logits that tie by the hundreds."""
    for vocab in (2000, 30000, 50257):
        x = draw(3, vocab, "f32", 1)
        x[0, 3::4096] += 50.0                       # the same place of every 4,096 (a thread's own elements)
        x[1, 8:8 + 24] += 40.0
        x[2] = x[2].round()
        for top in (5, 32):
            check(x, None, top, 1.0, logprobs(x, None, top, entropy=True))


@pytest.mark.parametrize("vocab", [6, 1000, 5000, 50257])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_rows_that_leave_little(vocab, kind):
    low = torch.finfo(KINDS[kind]).min
    x = draw(9, vocab, "f32", 2)
    x[0] = -INF
    x[1, 1:] = -INF                                 # one left
    x[2, 3:] = low                                  # masks of the type's lowest value
    x[3] = low
    x[4, vocab // 2] = NAN
    x[5, vocab // 2] = INF
    x[6] = NAN
    x[7, ::2] = -INF
    x[8, 0], x[8, 1] = low, -low                    # a difference past the largest number
    x = x.to(KINDS[kind])
    t = torch.tensor([0, 0, 1, 2, 0, 0, 0, 2, 1], device="cuda")
    for scale in (1.0, 0.5):
        got = logprobs(x, t, 5, scale, entropy=True)
        keep = [0, 1, 2, 3, 7] + ([8] if scale == 0.5 else [])
        check(x[keep], t[keep], 5, scale, type(got)(*(v[keep] for v in got)))
        assert got.logp[0] == -INF and got.entropy[0] == 0 and got.top_index[0].tolist() == [-1] * 5
        assert got.logp[1] == 0 and got.entropy[1] == 0 and got.top_index[1].tolist() == [0, -1, -1, -1, -1]
        assert bool(torch.isnan(got.logp[4:7]).all()) and bool(torch.isnan(got.entropy[4:7]).all())
        assert got.top_index[5, 0] == vocab // 2 and got.top_index[6].tolist() == [-1] * 5
        assert got.top_index[8, 0] == 1 and got.logp[8] == 0 and got.entropy[8] == 0
        g = torch.ones(9, device="cuda")
        d = logprobs_backward(g, x, t, got.stats, scale, got.entropy, g * 0.5)
        assert bool((d[0] == 0).all()) and bool(torch.isnan(d[4:7]).all())
        for i in (1, 2, 7, 8):
            want = O.logprobs_backward(host(x[i]), t[i].item(), 1.0, 0.5, scale) if i != 8 else np.zeros(vocab)
            assert near(host(d[i]), want, 1e-6 + HALF[kind] * np.abs(want))


def test_masked_rows_are_not_looked_at():
    x = torch.full((3, 3000), NAN, device="cuda")
    x[1] = draw(1, 3000, "f32", 1)
    t = torch.tensor([-100, 7, 3000], device="cuda")
    got = logprobs(x, t, 3, entropy=True)
    for i in (0, 2):
        assert got.logp[i] == 0 and got.entropy[i] == 0 and got.stats[i].tolist() == [0, 0]
        assert got.top_index[i].tolist() == [-1] * 3 and got.top_logp[i].tolist() == [0] * 3
    g = torch.full((3,), NAN, device="cuda")
    g[1] = 1.0
    d = logprobs_backward(g, x, t, got.stats, entropy=got.entropy, grad_entropy=g)
    assert bool((d[[0, 2]] == 0).all()) and bool(torch.isfinite(d[1]).all())


def check_backward(x, t, g, h, scale, kind, out=None):
    s32 = float(np.float32(scale))
    exact = [O.logprobs(r, None if t is None else k, 0, s32) for r, k in zip(host(x), [None] * len(x) if t is None else t.tolist())]
    stats = torch.tensor([e[2] for e in exact], dtype=torch.float32, device="cuda")
    entropy = torch.tensor([e[1] for e in exact], dtype=torch.float32, device="cuda")
    before = x.clone()
    got = logprobs_backward(g, x, t, stats, scale, None if h is None else entropy, h, out=out)
    for i in range(len(x)):
        target = None if t is None else int(t[i])
        gi, hi = (0.0 if v is None else float(v[i]) for v in (g, h))
        want = O.logprobs_backward(host(before[i]), target, gi, hi, s32)
        z = host(before[i]) * s32
        m, log_s = exact[i][2]
        logp = z - m - log_s
        p = np.exp(logp)
        terms = np.abs(gi) + np.abs(hi) * (np.abs(logp) + abs(exact[i][1]))
        slip = U * (4 * np.abs(logp) + abs(m) + abs(log_s))
        bound = s32 * p * (terms * (16 * U + slip) + np.abs(hi) * (slip + U * abs(exact[i][1]))) \
            + (U + HALF[kind] * (1 + 2 ** -6)) * np.abs(want)
        if target is not None and 0 <= target < len(z):
            bound[target] += 2 * U * s32 * abs(gi)
        assert np.all(np.abs(host(got[i]) - want) <= bound)
    return got


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("n,vocab", [(1, 1), (3, 2), (9, 7), (5, 100), (4, 1000), (3, 2049)])
def test_backward(n, vocab, kind):
    for extra, shift, scale in ((0, 0, 1.0), (3, 1, 0.7), (8, 0, 1.3)):
        x, t = draw(n, vocab, kind, vocab, extra, shift), draw_targets(n, vocab, 1)
        g, h = (torch.randn(n, generator=generator(s), device="cuda") for s in (2, 3))
        for grads in ((g, None), (g, h), (None, h)):
            first = check_backward(x, t, *grads, scale, kind)
            wide = torch.full((n, vocab + 5), 7.0, dtype=x.dtype, device="cuda")
            assert torch.equal(check_backward(x, t, *grads, scale, kind, out=wide[:, :vocab]), first)
            assert bool((wide[:, vocab:] == 7.0).all())
            again = x.clone()
            assert torch.equal(check_backward(again, t, *grads, scale, kind, out=again), first)      # in place
        check_backward(x, None, None, h, scale, kind)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("vocab,extra,pad", [(50257, 47, 0), (50257, 0, 0), (30522, 0, 6), (131072, 0, 0)])
def test_backward_of_long_rows(vocab, extra, pad, kind):
    """Against the formula in 64 bits on the device: rows and gradients of equal and of different alignment."""
    n = 6
    x, t = draw(n, vocab, kind, 5, extra), draw_targets(n, vocab, 6)
    g, h = (torch.randn(n, generator=generator(s), device="cuda") for s in (2, 3))
    got = logprobs(x, t, entropy=True)
    out = torch.full((n, vocab + pad), 7.0, dtype=x.dtype, device="cuda")
    logprobs_backward(g, x, t, got.stats, entropy=got.entropy, grad_entropy=h, out=out[:, :vocab])
    assert bool((out[:, vocab:] == 7.0).all())
    z = x.double().requires_grad_(True)
    logp = torch.log_softmax(z, 1)
    live = (t >= 0) & (t < vocab)
    total = (logp[torch.arange(n, device="cuda"), t.clamp(0, vocab - 1)] * g - (logp.exp() * logp).sum(1) * h) * live
    want, = torch.autograd.grad(total.sum(), z)
    with torch.no_grad():
        p = logp.exp()
        # p and log p from statistics that err by 250 u + 2 u log S; the entropy by 500 u times the mean of d and 300 u
        slip = U * (300 + 8 * logp.abs())
        bound = p * (g.abs()[:, None] + h.abs()[:, None] * (logp.abs() + 12)) * slip + p * h.abs()[:, None] * (slip + U * 9000) \
            + HALF[kind] * 1.02 * want.abs()
        bound[torch.arange(n), t.clamp(0, vocab - 1)] += 2 * U * g.abs()
        assert bool(((out[:, :vocab].double() - want).abs() <= bound).all())


def test_autograd_and_graphs():
    x, t = draw(6, 300, "f32", 1).contiguous().view(2, 3, 300).requires_grad_(True), draw_targets(6, 300, 2).view(2, 3)
    got = scored(x, t, top=4, scale=0.8, entropy=True)
    assert got.top_index.shape == (2, 3, 4) and not got.stats.requires_grad and not got.top_logp.requires_grad
    (-got.logp.mean() - 0.1 * got.entropy.sum()).backward()
    flat = x.detach().view(6, 300)
    one = torch.full((6,), 1.0, device="cuda")
    want = logprobs_backward(one / -6, flat, t.view(6), got.stats.view(6, 2), 0.8, got.entropy.detach().view(6), one * -0.1)
    assert torch.equal(x.grad.view(6, 300), want)
    x.grad = None
    scored(x, None, entropy=True).entropy.sum().backward()
    assert x.grad is not None
    x.grad = None
    scored(x, t).logp.sum().backward()
    assert x.grad is not None and bool((x.grad[0, 1] == 0).all())
    # a captured step
    logits, grad = draw(6, 5000, "bf16", 7), torch.ones(6, device="cuda")
    t = draw_targets(6, 5000, 3)
    eager = logprobs(logits, t, 3, entropy=True)
    d = logprobs_backward(grad, logits, t, eager.stats)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        again = logprobs(logits, t, 3, entropy=True)
        e = logprobs_backward(grad, logits, t, again.stats)
    for _ in range(2):
        [v.zero_() for v in (*again, e)]
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((*eager, d), (*again, e)))


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("scale", [2.0 ** -64, 1e-9, 30.0, 2.0 ** 64])
def test_extreme_scales(scale, kind):
    """Scales at which nothing differs, and at which only the largest is left; masked logits stay out of both."""
    x = draw(4, 3000, kind, 1)
    x[0, ::3] = -INF
    x[1, 1::2] = torch.finfo(KINDS[kind]).min
    x[2] = torch.arange(3000, device="cuda") % 7
    got = logprobs(x, None, 4, scale, entropy=True)
    check(x, None, 4, scale, got)
