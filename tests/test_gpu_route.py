"""Routing and its gradient on the GPU against the 64-bit oracle.

Bounds (u = 2^-24): a score is expf (2 ulp: 4u), a sum of at most 512 terms
added as 16 in a lane and 5 levels (21u) and a quotient: 27u; sigmoid less.
Renormalised: sum of at most 32 such (5 levels) and a quotient, times scale:
2 x 27u + 8u < 64u of the weight.  Choices are compared where the values that
they told apart differ by more than 1e-5, which is 1e-5 / 27u = 6 times the
score's error and the bias's rounding.
"""

import numpy as np
import pytest
import torch

from oracle import route as R
from reduction_reducer_gb300 import route, route_backward, routed

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
KINDS = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _device():
    torch.cuda.set_device(0)


def draw(T, E, dtype, seed=0, stride=None):
    gen = torch.Generator("cuda").manual_seed(seed)
    wide = torch.randn(max(T, 1), stride or E, generator=gen, device="cuda").mul_(1.5).to(KINDS[dtype])
    return wide[:T, :E]


def compare(x, got, k, mask=None, **how):
    index, weight = (t.cpu().numpy() for t in got)
    rows = x.double().cpu().numpy()
    bias = how.pop("bias", None)
    bias = None if bias is None else bias.double().cpu().numpy()
    compared = 0
    for t in range(len(rows)):
        if mask is not None and not mask[t]:
            assert (index[t] == -1).all() and (weight[t] == 0).all()
            continue
        want, w, margin = R.route_token(rows[t], k, bias=bias, **how)
        if margin <= 1e-5:
            continue
        compared += 1
        assert index[t].tolist() == want, t
        assert np.all(np.abs(weight[t] - w) <= 64 * U * np.abs(w)), t
    return compared


SHAPES = [(1, 1, 1), (5, 8, 2), (33, 32, 8), (7, 33, 4), (300, 60, 4), (40, 64, 6), (65, 128, 8), (20, 200, 12),
          (257, 256, 8), (19, 300, 32), (9, 512, 10)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k", SHAPES)
def test_route(T, E, k, score, renorm, dtype):
    x = draw(T, E, dtype, seed=E)
    how = dict(score=score, renorm=renorm, scale=2.5)
    assert compare(x, route(x, k, **how), k, **how) >= 0.6 * T
    bias = torch.randn(E, device="cuda") * 0.3
    assert compare(x, route(x, k, bias=bias, **how), k, bias=bias, **how) >= 0.6 * T


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups,top,k", [(8, 8, 3, 3), (8, 2, 1, 4), (64, 8, 4, 6), (72, 8, 3, 8), (60, 4, 2, 5),
                                            (256, 8, 4, 8), (256, 32, 5, 8), (512, 16, 16, 10), (33, 11, 4, 2)])
def test_groups(E, groups, top, k, score):
    x = draw(130, E, "f32", seed=E + groups)
    bias = torch.randn(E, device="cuda") * 0.1
    for b in (None, bias):
        how = dict(score=score, renorm=True, groups=groups, top_groups=top)
        compared = compare(x, route(x, k, bias=b, **how), k, bias=b, **how)
        assert compared >= 0.5 * 130


def test_ties_go_to_the_lowest():
    for E in (5, 64, 300):
        x = torch.zeros(3, E, device="cuda")
        x[1] = -0.0
        x[2, ::2] = -0.0                                             # -0 and +0 are equal
        for how in (dict(), dict(score="sigmoid", bias=torch.zeros(E, device="cuda"))):
            index, w = route(x, 4, **how)
            assert index.tolist() == [[0, 1, 2, 3]] * 3
    x = torch.zeros(1, 32, device="cuda")
    x[0, 9:12] = 1.0
    assert route(x, 5)[0].tolist() == [[9, 10, 11, 0, 1]]
    # groups that tie: the lowest ones
    index, _ = route(torch.zeros(1, 32, device="cuda"), 3, score="sigmoid", groups=8, top_groups=2)
    assert index.tolist() == [[0, 1, 2]]
    # bf16 logits tie often; every row against the oracle, whose margin leaves exact ties in
    x = (torch.randn(200, 64, generator=torch.Generator("cuda").manual_seed(3), device="cuda") * 4).round().bfloat16()
    for how in (dict(score="softmax"), dict(score="sigmoid", bias=torch.zeros(64, device="cuda"))):
        assert compare(x, route(x, 6, **how), 6, **how) > 100


def test_rows_that_leave_nothing():
    inf, nan = float("inf"), float("nan")
    x = torch.tensor([[-inf] * 6, [-inf, 2.0, -inf, 1.0, -inf, -inf], [0.0, nan, 1.0, 2.0, 3.0, 4.0],
                      [0.0, inf, 1.0, 2.0, 3.0, 4.0], [nan] * 6, [torch.finfo(torch.float32).min] * 6], device="cuda")
    for dtype in KINDS.values():
        index, w = route(x.to(dtype), 3, score="softmax", renorm=True)
        assert index[0].tolist() == [-1, -1, -1] and w[0].tolist() == [0, 0, 0]
        assert index[1].tolist() == [1, 3, -1] and w[1, 2] == 0
        assert torch.allclose(w[1, :2].cpu(), torch.softmax(torch.tensor([2.0, 1.0]), 0), rtol=1e-6)
        assert index[2].tolist() == [5, 4, 3] and bool(torch.isnan(w[2]).all())
        assert bool(torch.isnan(w[3]).all()) and bool(torch.isnan(w[4]).all()) and index[4].tolist() == [-1, -1, -1]
        if dtype == torch.float32:                                   # the type's lowest value is a value
            assert index[5].tolist() == [0, 1, 2] and torch.allclose(w[5], torch.full((3,), 1 / 3, device="cuda"))
        index, w = route(x.to(dtype), 3, score="sigmoid")
        assert index[0].tolist() == [-1] * 3 and index[3].tolist() == [1, 5, 4] and w[3, 0] == 1.0
        assert bool(torch.isnan(w[2]).all()) and w[5, 0] == 0.0
        g = torch.ones(6, 3, device="cuda")
        for score in ("softmax", "sigmoid"):
            for renorm in (False, True):
                index, w = route(x.to(dtype), 3, score=score, renorm=renorm)
                d = route_backward(g, x.to(dtype), index, w, score=score, renorm=renorm)
                assert bool((d[0] == 0).all()) and bool((d[1, [0, 2, 4, 5]] == 0).all())
                assert bool(torch.isfinite(d[1]).all())
    # an expert barred by its bias, and a group of barred ones
    x = draw(40, 16, "f32")
    bias = torch.zeros(16, device="cuda")
    bias[3] = -inf
    assert not bool((route(x, 5, score="sigmoid", bias=bias)[0] == 3).any())
    bias[4:8] = -inf
    index, _ = route(x, 5, score="sigmoid", bias=bias, groups=4, top_groups=2)
    assert not bool(((index >= 3) & (index < 8)).any())


def test_mask_counts_and_stride():
    T, E, k = 1000, 96, 6
    x = draw(T, E, "bf16", stride=131)
    mask = torch.rand(T, device="cuda") < 0.7
    x[~mask] = float("nan")                                          # never looked at
    counts = torch.full((E,), 5, dtype=torch.int32, device="cuda")
    how = dict(score="softmax", renorm=True)
    got = route(x, k, mask=mask, counts=counts, **how)
    compare(x, got, k, mask=mask.cpu().numpy(), **how)
    chosen = got[0][mask].flatten().long()
    assert torch.equal(counts.long() - 5, torch.bincount(chosen, minlength=E))
    route(x, k, mask=mask.to(torch.uint8), counts=counts, **how)     # added to
    assert torch.equal(counts.long() - 5, 2 * torch.bincount(chosen, minlength=E))
    none = route(x, k, mask=torch.zeros_like(mask), counts=counts, **how)
    assert bool((none[0] == -1).all()) and bool((none[1] == 0).all())
    g = torch.randn(T, k, device="cuda")
    for s in ("softmax", "sigmoid"):
        for renorm in (False, True):
            index, w = route(x, k, mask=mask, score=s, renorm=renorm)
            d = route_backward(g, x, index, w, score=s, renorm=renorm)
            assert bool((d[~mask] == 0).all()) and bool(torch.isfinite(d).all())


def test_no_tokens():
    x = torch.empty(0, 16, device="cuda")
    index, w = route(x, 2)
    assert index.shape == (0, 2) and w.shape == (0, 2)
    assert route_backward(w, x, index, w).shape == (0, 16)


def test_many_tokens():
    """More tokens than the grid's warps: every row as in the plain order, counts whole."""
    T, E, k = 40_003, 40, 5
    x = draw(T, E, "f32")
    counts = torch.zeros(E, dtype=torch.int32, device="cuda")
    index, w = route(x, k, counts=counts)
    want = x.sort(dim=1, descending=True, stable=True).indices[:, :k]
    assert torch.equal(index.long(), want)
    assert torch.equal(counts.long(), torch.bincount(want.flatten(), minlength=E))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k", SHAPES)
def test_backward(T, E, k, score, renorm, dtype):
    x = draw(T, E, dtype, seed=T)
    how = dict(score=score, renorm=renorm, scale=2.5)
    index, w = route(x, k, **how)
    g = torch.randn(T, k, generator=torch.Generator("cuda").manual_seed(1), device="cuda")
    wide = torch.full((T, E + 3), 7.0, dtype=x.dtype, device="cuda")
    d = route_backward(g, x, index, w, out=wide[:, :E], **how)
    assert bool((wide[:, E:] == 7.0).all())
    got, rows = d.double().cpu().numpy(), x.double().cpu().numpy()
    for t in range(min(T, 40)):
        want = R.backward_token(rows[t], index[t].tolist(), g[t].cpu().numpy(), score, renorm, 2.5)
        # terms: weights (64u), g w summed over k, and for softmax a score times their sum
        size = np.abs(g[t].cpu().numpy() * w[t].cpu().numpy()).sum()
        bound = 160 * U * size + (2.0 ** -8 * np.abs(want) if dtype == "bf16" else 0)
        assert np.all(np.abs(got[t] - want) <= bound), t


@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("scale", [1.0, -2.0, 1e-30, 1e38])
def test_backward_where_the_first_weight_says_little(scale, renorm):
    """Sigmoid scores of a token over the whole range, the first slot's zero or the smallest (the bias puts it first),
    and weights near the ends of fp32's range."""
    T, E, k = 64, 24, 6
    x = draw(T, E, "f32", seed=11) * 6.0
    bias = torch.zeros(E, device="cuda")
    bias[2:5] = 3.0
    x[:16, 2] = -200.0
    x[16:32, 2] = -60.0
    x[8:24, 3:5] = -150.0
    x[32:40] = -120.0
    x[40:48, 7] = 90.0
    index, w = route(x, k, score="sigmoid", bias=bias, renorm=renorm, scale=scale)
    g = torch.randn(T, k, generator=torch.Generator("cuda").manual_seed(1), device="cuda") * 0.1
    d = route_backward(g, x, index, w, score="sigmoid", renorm=renorm, scale=scale).double().cpu().numpy()
    rows = x.double().cpu().numpy()
    for t in range(T):
        gt = g[t].double().cpu().numpy()
        if not bool((w[t] != 0).any()):                              # scores below fp32's least number
            assert np.all(d[t] == 0), t
            continue
        want = R.backward_token(rows[t], index[t].tolist(), gt, "sigmoid", renorm, scale)
        size = np.abs(gt * w[t].double().cpu().numpy()).sum()
        assert np.all(np.abs(d[t] - want) <= 160 * U * size + 2.0 ** -140), t


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_backward_against_differences(score, renorm):
    """The kernel's gradient against central differences of the kernel's own weights at a choice that stays: a step of
    2^-6 errs by its square over 6 times third derivatives of at most 1 / 8 x scale (2^-12 / 48 x 2.5 < 1.3e-5 a slot)
    and by the weights' 64u over the step (64 x 2^-24 x 2.5 / 2^-6 < 6.2e-4)."""
    E, k, h = 12, 3, 2.0 ** -6
    x = torch.randn(1, E, generator=torch.Generator("cuda").manual_seed(5), device="cuda")
    x[0, [2, 7, 9]] += 5.0                                           # a choice that no small step changes
    g = torch.tensor([[0.5, -1.0, 2.0]], device="cuda")
    how = dict(score=score, renorm=renorm, scale=2.5)
    index, w = route(x, k, **how)
    d = route_backward(g, x, index, w, **how)[0].cpu()
    for i in range(E):
        up, down = x.clone(), x.clone()
        up[0, i] += h
        down[0, i] -= h
        (iu, wu), (id_, wd) = route(up, k, **how), route(down, k, **how)
        at_u = {int(e): float(v) for e, v in zip(iu[0], wu[0])}
        at_d = {int(e): float(v) for e, v in zip(id_[0], wd[0])}
        assert set(at_u) == set(at_d) == {2, 7, 9}
        slope = sum(float(gr) * (at_u[int(e)] - at_d[int(e)]) / (2 * h) for gr, e in zip(g[0], index[0]))
        assert abs(slope - float(d[i])) <= 3.5 * (1.3e-5 + 6.2e-4)


def test_autograd():
    x = draw(50, 24, "f32").clone().requires_grad_(True)
    target = torch.randn(50, 4, device="cuda")
    index, w = routed(x, 4, score="sigmoid", renorm=True, scale=2.0)
    ((w - target) ** 2).sum().backward()
    y = x.detach().clone().requires_grad_(True)
    s = torch.sigmoid(y).gather(1, index.long())
    ((s / s.sum(1, keepdim=True) * 2.0 - target) ** 2).sum().backward()
    assert torch.allclose(x.grad, y.grad, rtol=1e-4, atol=1e-6)
    assert not index.requires_grad


def test_no_second_derivative():
    x = draw(9, 16, "f32").requires_grad_(True)
    _, w = routed(x, 4)
    d, = torch.autograd.grad((w ** 2).sum(), x, create_graph=True)
    with pytest.raises(RuntimeError):
        torch.autograd.grad(d.sum(), x)


def test_other_stream():
    x = draw(500, 64, "f32")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = (torch.empty(500, 4, dtype=torch.int32, device="cuda"), torch.empty(500, 4, device="cuda"))
    route(x, 4, out=out, stream=side)
    side.synchronize()
    assert torch.equal(out[0], route(x, 4)[0]) and torch.equal(out[1], route(x, 4)[1])


def test_outputs_are_memory_of_their_stream():
    """The allocator may hand out, on the current stream, memory that kernels queued there still use: what a call on
    another stream writes into comes from that stream's."""
    x, g = draw(500, 64, "f32"), torch.ones(500, 4, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())

    def owner(t):
        p = t.data_ptr()
        return [s["stream"] for s in torch.cuda.memory_snapshot()
                if s["address"] <= p < s["address"] + s["total_size"]][0]

    for stream in (side, side.cuda_stream):
        index, w = route(x, 4, stream=stream)
        d = route_backward(g, x, index, w, stream=stream)
        assert [owner(t) for t in (index, w, d)] == [side.cuda_stream] * 3
        torch.cuda.synchronize()
        assert torch.equal(index, route(x, 4)[0])


def test_refusals_of_tensors():
    x = draw(4, 8, "f32")
    with pytest.raises(ValueError):
        route(x.half(), 2)
    with pytest.raises(ValueError):
        route(x.t(), 2)
    with pytest.raises(ValueError):
        route(x, 2, score="tanh")
    with pytest.raises(ValueError):
        route(x, 2, bias=torch.zeros(7, device="cuda"))
    with pytest.raises(ValueError):
        route(x, 2, counts=torch.zeros(8, device="cuda"))
    with pytest.raises(ValueError):
        route(x, 2, mask=torch.zeros(5, dtype=torch.bool, device="cuda"))
    with pytest.raises(ValueError):
        route(x, 2, out=(torch.zeros(4, 2, device="cuda"), torch.zeros(4, 2, device="cuda")))
    from reduction_reducer_gb300 import InvalidArg
    with pytest.raises(InvalidArg):
        route(x, 9)
    with pytest.raises(InvalidArg):
        route(x, 2, groups=3)


def test_a_bias_that_ends_at_a_power_of_two():
    """score + bias just below 2, where a rounded key would be that of 2: still the best."""
    for bias in (1 - 2.0 ** -23, 1 - 2.0 ** -24, 1.0, 3 - 2.0 ** -22, 2.0 ** 19 - 1):
        x = draw(6, 16, "f32", seed=3)
        x[:, 5] = 40.0
        b = torch.zeros(16, device="cuda")
        b[5] = bias
        index, _ = route(x, 3, score="sigmoid", bias=b)
        assert bool((index[:, 0] == 5).all()), bias
        assert torch.equal(index.long(), fp32_choice(x, 3, "sigmoid", b))
        b[5] = -bias
        assert torch.equal(route(x, 3, score="sigmoid", bias=b)[0].long(), fp32_choice(x, 3, "sigmoid", b))


@pytest.mark.parametrize("E,groups,top,k", [(500, 10, 4, 8), (480, 12, 3, 6), (510, 30, 7, 8)])
def test_counts_where_the_groups_do_not_fit_the_lanes(E, groups, top, k):
    """Groups that waste so many slots that every token is chosen by the definition: with a bias, the counts and the
    choice stay whole."""
    x = draw(700, E, "f32", seed=E)
    bias = torch.randn(E, generator=torch.Generator("cuda").manual_seed(1), device="cuda") * 0.1
    counts = torch.zeros(E, dtype=torch.int32, device="cuda")
    index, _ = route(x, k, score="sigmoid", bias=bias, groups=groups, top_groups=top, counts=counts)
    assert torch.equal(index.long(), fp32_choice(x, k, "sigmoid", bias, groups, top))
    assert torch.equal(counts.long(), torch.bincount(index.flatten().long(), minlength=E))


def fp32_choice(x, k, score, bias, groups=1, top_groups=1):
    """The choice by the definition in fp32, step by step: exponentials, products and sums as torch rounds them."""
    x = x.float()
    s = 1 / (1 + torch.exp(-x)) if score == "sigmoid" else x
    c = s + bias
    if groups > 1:
        T, E = x.shape
        worth = c.view(T, groups, E // groups).topk(min(2, E // groups)).values.sum(2)
        first = worth.argsort(dim=1, descending=True, stable=True)[:, :top_groups]
        stay = torch.zeros(T, groups, dtype=torch.bool, device="cuda").scatter_(1, first, True)
        c = torch.where(stay.repeat_interleave(E // groups, dim=1), c, float("-inf"))
    return c.argsort(dim=1, descending=True, stable=True)[:, :k]


@pytest.mark.parametrize("E", [8, 24, 64, 128, 256, 320, 512])
@pytest.mark.parametrize("spread", [0.0, 6e-8, 1e-6, 1e-4])
def test_near_ties_are_decided_by_the_fp32_definition(E, spread):
    """A bias that brings all experts of the first row within `spread` of one another: no two keys, or all, tell them
    apart; the fp32 sums do, and equal sums go to the lowest expert."""
    gen = torch.Generator("cuda").manual_seed(E)
    x = torch.randn(1, E, generator=gen, device="cuda") + torch.randn(50, 1, generator=gen, device="cuda") * 1e-3
    bias = 0.7 - torch.sigmoid(x[0]) + torch.rand(E, generator=gen, device="cuda") * spread
    for k in (1, 4, 8):
        index, _ = route(x, k, score="sigmoid", bias=bias)
        assert torch.equal(index.long(), fp32_choice(x, k, "sigmoid", bias)), k
    for groups, top in ((4, 2), (8, 3)):
        index, _ = route(x, 2, score="sigmoid", bias=bias, groups=groups, top_groups=top)
        assert torch.equal(index.long(), fp32_choice(x, 2, "sigmoid", bias, groups, top))
    # logits themselves a few ulps apart
    y = 1.0 + torch.randint(0, 5, (50, E), generator=gen, device="cuda") * 2.0 ** -23
    for k in (1, 4, 8):
        assert torch.equal(route(y, k)[0].long(), y.argsort(dim=1, descending=True, stable=True)[:, :k])


@pytest.mark.parametrize("scale", [0.5, 3.0, 100.0, 1e5, 1e8])
def test_biases_of_any_range(scale):
    gen = torch.Generator("cuda").manual_seed(2)
    x = torch.randn(60, 96, generator=gen, device="cuda")
    bias = torch.randn(96, generator=gen, device="cuda") * scale
    for groups, top in ((1, 1), (8, 3)):
        index, _ = route(x, 6, score="sigmoid", bias=bias, groups=groups, top_groups=top)
        assert torch.equal(index.long(), fp32_choice(x, 6, "sigmoid", bias, groups, top))


@pytest.mark.parametrize("E,k", [(64, 7), (128, 8), (256, 16), (512, 12), (512, 32)])
def test_all_the_best_next_to_one_another(E, k):
    """Sorted logits: one lane holds every expert that is chosen."""
    x = torch.linspace(3, -3, E, device="cuda").repeat(20, 1)
    x[1::2] = x[1::2].flip(1)
    want = x.argsort(dim=1, descending=True, stable=True)[:, :k]
    assert torch.equal(route(x, k)[0].long(), want)
    zero = torch.zeros(E, device="cuda")
    assert torch.equal(route(x, k, score="sigmoid", bias=zero)[0].long(), fp32_choice(x, k, "sigmoid", zero))


@pytest.mark.parametrize("E,groups,top,k", [(510, 3, 2, 5), (510, 30, 7, 8), (96, 32, 9, 12), (512, 32, 3, 20)])
def test_groups_of_odd_sizes(E, groups, top, k):
    gen = torch.Generator("cuda").manual_seed(E + groups)
    x = torch.randn(90, E, generator=gen, device="cuda")
    bias = torch.randn(E, generator=gen, device="cuda") * 0.1
    index, _ = route(x, k, score="sigmoid", bias=bias, groups=groups, top_groups=top)
    assert torch.equal(index.long(), fp32_choice(x, k, "sigmoid", bias, groups, top))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("E,k", [(64, 7), (64, 12), (100, 4), (128, 8), (130, 3), (200, 14), (256, 8), (256, 16)])
def test_more_than_a_million_logits(E, k, dtype):
    """Batches large enough for every layout, against the fp32 definition: ordinary rows, rows of near ties, sorted
    ones, masked ones and ones that are not numbers, mixed within warps."""
    T = (1 << 20) // E + 37
    gen = torch.Generator("cuda").manual_seed(E * k)
    x = torch.randn(T, E, generator=gen, device="cuda") * 1.5
    x[1::7] = 1.0 + torch.randint(0, 4, x[1::7].shape, generator=gen, device="cuda") * 2.0 ** -23
    x[2::7] = torch.linspace(3, -3, E, device="cuda")
    x[3::11] = x[3::11].round()                                      # exact ties
    x = x.to(KINDS[dtype])
    mask = torch.rand(T, generator=gen, device="cuda") < 0.9
    x[~mask] = float("nan")
    x[5::301] = float("-inf")
    x[6::301, : E - 2] = float("-inf")
    x[7::301, 3] = float("nan")
    bias = torch.randn(E, generator=gen, device="cuda") * 0.2
    live = mask.clone()
    live[7::301] = False                                             # NaN weights: checked by themselves
    y = torch.where(torch.isnan(x), float("-inf"), x.float())
    for score, b in (("softmax", None), ("sigmoid", bias), ("sigmoid", None)):
        counts = torch.zeros(E, dtype=torch.int32, device="cuda")
        index, w = route(x, k, score=score, bias=b, renorm=True, mask=mask, counts=counts)
        c = y if b is None else torch.where(y > float("-inf"), 1 / (1 + torch.exp(-y)) + b, float("-inf"))
        order = c.argsort(dim=1, descending=True, stable=True)[:, :k]
        want = torch.where(c.gather(1, order) > float("-inf"), order, -1)
        assert torch.equal(index.long()[live], want[live])
        assert bool((index[~mask] == -1).all()) and bool((w[~mask] == 0).all())
        assert bool(torch.isnan(w[7::301][mask[7::301]]).all())
        chosen = index[index >= 0].long()
        assert torch.equal(counts.long(), torch.bincount(chosen, minlength=E))
        d = y.double()
        s = torch.sigmoid(d) if score == "sigmoid" else torch.exp(d - d.amax(1, keepdim=True).clamp(min=-1e30))
        s = torch.where(index >= 0, s.gather(1, index.clamp(min=0).long()), 0.0)
        total = s.sum(1, keepdim=True)
        ref = torch.where(total > 0, s / total, 0.0)
        assert bool(((w.double() - ref).abs()[live] <= 64 * U * ref[live]).all())


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_softmax_with_a_bias_and_many_tokens(score):
    """Against the 64-bit scores where these tell the experts apart by more than the bound of a score, 27u, twice."""
    T, E, k = 9000, 256, 8
    gen = torch.Generator("cuda").manual_seed(8)
    x = torch.randn(T, E, generator=gen, device="cuda")
    bias = torch.randn(E, generator=gen, device="cuda") * 0.01
    for groups, top in ((1, 1), (8, 4)):
        index, w = route(x, k, score=score, bias=bias, groups=groups, top_groups=top)
        s = torch.softmax(x.double(), 1) if score == "softmax" else torch.sigmoid(x.double())
        c = s + bias.double()
        clear = torch.ones(T, dtype=torch.bool, device="cuda")
        if groups > 1:
            worth = c.view(T, groups, -1).topk(2).values.sum(2)
            ranked = worth.sort(dim=1, descending=True)
            clear &= ranked.values[:, top - 1] - ranked.values[:, top] > 1e-5
            stay = torch.zeros(T, groups, dtype=torch.bool, device="cuda").scatter_(1, ranked.indices[:, :top], True)
            c = torch.where(stay.repeat_interleave(E // groups, dim=1), c, -9.0)
        ranked = c.sort(dim=1, descending=True)
        clear &= (ranked.values[:, :k] - ranked.values[:, 1:k + 1]).amin(1) > 1e-5
        assert float(clear.float().mean()) > 0.5
        assert torch.equal(index.long()[clear], ranked.indices[:, :k][clear])
        ref = s.gather(1, index.long())
        assert bool(((w.double() - ref).abs() <= 64 * U * ref).all())


def test_offsets_past_32_bits():
    """8,388,613 tokens over 256 experts: logits, and their gradient, of more than 2^31 elements."""
    T, E, k = (1 << 23) + 5, 256, 2
    x = torch.zeros(T, E, dtype=torch.bfloat16, device="cuda")
    x[-3:, 200] = 2.0
    x[-3:, 17] = 1.0
    counts = torch.zeros(E, dtype=torch.int32, device="cuda")
    index, w = route(x, k, renorm=True, counts=counts)
    assert index[-3:].tolist() == [[200, 17]] * 3 and index[:-3].unique().tolist() == [0, 1]
    assert int(counts.sum()) == 2 * T and counts[[0, 1, 17, 200]].tolist() == [T - 3, T - 3, 3, 3]
    s = torch.softmax(torch.tensor([2.0, 1.0]), 0)
    assert torch.allclose(w[-3:].cpu(), s.repeat(3, 1), rtol=64 * U) and torch.equal(w[:-3], torch.full((T - 3, 2), 0.5, device="cuda"))
    g = torch.zeros(T, k, device="cuda")
    g[-1, 0] = 1.0
    for renorm in (True, False):
        if not renorm:
            index, w = route(x, k)
        d = route_backward(g, x, index, w, renorm=renorm)
        assert int((d[:-1] != 0).sum()) == 0
        want = R.backward_token(x[-1].double().cpu().numpy(), [200, 17], [1.0, 0.0], "softmax", renorm, 1.0)
        assert np.all(np.abs(d[-1].double().cpu().numpy() - want) <= 2.0 ** -8 * np.abs(want) + 160 * U)
