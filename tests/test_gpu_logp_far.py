"""The logits' gradient of rows whose largest logit times scale is far from zero, or past the fp32 range, with the
statistics that the forward pass gave.

Bounds (u = 2^-24).  Statistics: log S errs by 250 u + 2 u log S, and by one more step of its own (2 u log S) where its last
bit says which of two numbers m is; m is exact where |scale m| is above 64, and below that the product's rounding, at most
64 u, is the error of log p.  The difference, its scale and base are 4 u |z - m|, log p's own rounding u |log p|, 2^x 8 u:
p errs by slip = u (322 + 8 |log p| + 8 log S) of itself.  The factor g + h (log p + H) errs by 16 u of its terms and |h| of
slip and the entropy's 250 u + 500 u |H - log S| + 4 u H.  A target adds 2 u |g|, the result its own rounding, and what is
below 2^-126 may be zero."""

import pytest
import torch

from reduction_reducer_gb300 import logprobs, logprobs_backward, scored

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
KINDS = {"f32": torch.float32, "bf16": torch.bfloat16}
HALF = {"f32": U, "bf16": 2.0 ** -8}
INF = float("inf")


@pytest.fixture(scope="module", autouse=True)
def _device():
    torch.cuda.set_device(0)


def rows(vocab, kind, seed=0):
    """(logits, targets): masked rows, rows with an offset, rows of the largest numbers."""
    gen = torch.Generator("cuda").manual_seed(seed)
    low, high = torch.finfo(KINDS[kind]).min, torch.finfo(KINDS[kind]).max
    noise = torch.randn(19, vocab, generator=gen, device="cuda") * 2
    x, t = noise.clone(), torch.randint(vocab, (19,), generator=gen, device="cuda")
    x[0], x[1], x[2], x[3] = low, -1e9, -1e4, high
    x[4:7] += torch.tensor([1e4, -1e4, 100.0], device="cuda")[:, None]
    x[7] = low
    x[7, ::2] = low / 2
    x[8, 3] = x[9, 3] = high
    t[8], t[9] = 3, 1                                      # the largest itself, and one that is nothing beside it
    x[10] = -INF
    x[10, :5] = low
    x[11] = -1e9 + 64 * noise[11].round()
    x[12:15] = -INF
    x[12, 2] = x[13, 2] = low
    t[12], t[13] = 2, 0
    x[15] = 1e20 * (1 + U * noise[15].round())
    x[16] -= 70
    x[17] += 60
    x[18] -= 1e6
    return x.to(KINDS[kind]), t


def gradient64(x, t, g, h, scale):
    """The formula, log p, log S and the entropy; a row of nothing has no gradient."""
    z = x.double() * scale
    m = z.amax(1, keepdim=True)
    some = m > -INF
    d = torch.where(some, z - torch.where(some, m, 0.0), -INF)
    e = torch.exp(d)
    total = torch.where(some, e.sum(1, keepdim=True), 1.0)
    logp = d - total.log()
    p = torch.exp(logp)
    entropy = total.log() - (e * torch.where(e > 0, d, 0.0)).sum(1, keepdim=True) / total
    hot = torch.nn.functional.one_hot(t, x.shape[1]).double()
    logp = torch.where(p > 0, logp, 0.0)
    want = scale * (g[:, None] * (hot - p) - h[:, None] * p * (logp + entropy))
    return torch.where(some, want, 0.0), p, logp, total.log(), entropy, hot


def check(got, x, t, g, h, scale, kind, more=0.0):
    want, p, logp, log_s, entropy, hot = gradient64(x, t, g, h, scale)
    slip = U * (322 + 8 * logp.abs() + 8 * log_s) + more
    g, h = g.double().abs()[:, None], h.double().abs()[:, None]
    off = U * (250 + 500 * (entropy - log_s).abs() + 4 * entropy.abs())
    bound = scale * p * ((g + h * (logp.abs() + entropy)) * (16 * U + slip) + h * (slip + off)) + 2 * U * scale * g * hot \
        + (U + HALF[kind] * (1 + 2 ** -6)) * want.abs() + scale * (g + 200 * h) * 2.0 ** -126
    wrong = ~((got.double() - want).abs() <= bound)
    assert not bool(wrong.any()), (wrong.any(1).nonzero().flatten().tolist(), got[wrong][:4], want[wrong][:4])


def f32(x):
    return float(torch.tensor(x, dtype=torch.float32))


SCALES = [1.0, 2.0, 1 / 0.7, 1 / 1.3, 0.3, 1.9, 2.0 ** -64 * 1.3, 2.0 ** 64]


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("vocab", [7, 1000, 5000, 50257])
@pytest.mark.parametrize("scale", SCALES)
def test_gradient(scale, vocab, kind):
    x, t = rows(vocab, kind)
    gen = torch.Generator("cuda").manual_seed(1)
    g, h = (torch.randn(len(x), generator=gen, device="cuda") for _ in range(2))
    zero = torch.zeros_like(g)
    forward = logprobs(x, t, scale=scale, entropy=True)
    for by, of in ((g, zero), (g, h), (zero, h)):
        entropy = forward.entropy if of is h else None
        got = logprobs_backward(by, x, t, forward.stats, scale, entropy, of if of is h else None)
        check(got, x, t, by, of, f32(scale), kind)
        again = x.clone()
        assert torch.equal(logprobs_backward(by, again, t, forward.stats, scale, entropy, of if of is h else None, out=again), got)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("vocab", [6, 3000, 20000])
@pytest.mark.parametrize("scale", [0.5, 0.3, 2.0 ** -64, 2.0 ** -40 * 1.7])
def test_differences_past_the_largest_number(scale, vocab, kind):
    """The type's largest and lowest in one row: their difference is no fp32 number, and its product with scale is.  It errs
    by 2 u (two products of different signs, added: 1 u each) and log S, which nothing else in the row adds to, is log 3."""
    low = torch.finfo(KINDS[kind]).min
    x = torch.full((2, vocab), -INF, dtype=KINDS[kind], device="cuda")
    x[:, :3], x[:, 3] = -low, low
    t = torch.tensor([3, 1], device="cuda")
    got = logprobs(x, t, 5, scale, entropy=True)
    log3 = torch.tensor(3.0, dtype=torch.float64).log().item()
    far = 2 * low * f32(scale)
    for value, want in ((got.logp[0], far), (got.top_logp[0, 3], far), (got.top_logp[1, 3], far), (got.logp[1], -log3),
                        (got.top_logp[0, 0], -log3), (got.entropy[0], log3)):
        assert abs(float(value) - want) <= 4 * U * abs(want) + 20 * U, (float(value), want)
    assert got.top_index[0].tolist() == [0, 1, 2, 3, -1] and float(got.top_logp[0, 4]) == -INF


@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_many_largest_logits(kind):
    """Every m of a binade and its neighbours, two of which may have the same product with scale."""
    gen = torch.Generator("cuda").manual_seed(3)
    n = 20000
    m = torch.exp2(torch.rand(n, generator=gen, device="cuda") * 60 + 4) * (1 - 2 * (torch.rand(n, generator=gen, device="cuda") < 0.5))
    x = torch.stack([m, m - m.abs(), m - 3, m - 0.25, -INF + m], 1).to(KINDS[kind])
    t = torch.full((n,), 3, device="cuda")
    one, none = torch.ones(n, device="cuda"), torch.zeros(n, device="cuda")
    for scale in (1.0, 1 / 0.7, 1 / 1.3, 1.999999, 1.0000001, 37.5):
        got = logprobs_backward(one, x, t, logprobs(x, t, scale=scale).stats, scale)
        check(got, x, t, one, none, f32(scale), kind)


@pytest.mark.parametrize("scale", [1 / 0.7, 1 / 1.3])
def test_statistics_from_elsewhere(scale):
    """With fp32 statistics that were made from the definition: which of two numbers m is, is not told, and log p may be off
    by a step of scale m more (2 u of it)."""
    x, t = rows(1000, "f32")
    x, t = x[[4, 5, 6, 16, 17, 18]], t[[4, 5, 6, 16, 17, 18]]
    z = x.double() * f32(scale)
    m = z.amax(1, keepdim=True)
    stats = torch.cat([m, torch.exp(z - m).sum(1, keepdim=True).log()], 1).float()
    one, none = torch.ones(len(x), device="cuda"), torch.zeros(len(x), device="cuda")
    check(logprobs_backward(one, x, t, stats, scale), x, t, one, none, f32(scale), "f32", more=2 * U * m.abs())


@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_masked_rows_under_autograd(kind):
    """A row that a mask of the type's lowest value fills is uniform, at any temperature."""
    x = torch.full((3, 4, 3001), torch.finfo(KINDS[kind]).min, dtype=KINDS[kind], device="cuda")
    x[1, 2, :7] = 1.0
    x.requires_grad_(True)
    t = torch.zeros(3, 4, dtype=torch.int64, device="cuda")
    for temperature in (0.5, 0.7, 1.0, 1.3):
        got = scored(x, t, scale=1 / temperature, entropy=True)
        grad, = torch.autograd.grad(got.logp.sum(), x)
        one, flat = torch.ones(12, device="cuda"), x.detach().view(12, 3001)
        check(grad.view(12, 3001), flat, t.view(12), one, 0 * one, f32(1 / temperature), kind)
