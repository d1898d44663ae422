"""Layer norm and its gradient on the GPU against the 64-bit oracle.

Bounds (u = 2^-24, h = half a step of the result's type).  A sum over a row
has chains of c = max(48, dim / 1024 + 24) additions at most.  The mean errs by
(c + 1) u mean|x|, which enters y times r |w|; the variance by (c + 4) u of itself
and the square of the mean's error, so r by (c + 8) u and (mean's error r)^2;
products, bias and rounding are 4 u and h.  The gradient takes the statistics as
given: xh errs by 3 u, the two means by (c + 4) u of the mean magnitudes, the
difference and product by 4 u of each term.  The parameters' gradients add
rows terms in a thread and 64 more parts' sums: (rows + 80) u of the magnitudes."""

import numpy as np
import pytest
import torch

from oracle import tokens as O
from reduction_reducer_gb300 import layer_norm, layer_norm_backward, layer_normed

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
KINDS = {"f32": torch.float32, "bf16": torch.bfloat16}
HALF = {"f32": U, "bf16": 2.0 ** -8}
DIMS = [1, 3, 4, 8, 60, 64, 72, 100, 128, 129, 136, 256, 264, 512, 769, 1000, 1004, 1023, 1024, 1032, 2048, 2500, 4096, 4104, 8200, 11101, 16384, 33000]


@pytest.fixture(scope="module", autouse=True)
def _device():
    torch.cuda.set_device(0)


def generator(seed):
    return torch.Generator("cuda").manual_seed(seed)


def rows(n, dim, kind, seed, extra=0, shift=0, offset=0.7):
    flat = torch.randn(max(n, 1) * (dim + extra) + shift, generator=generator(seed), device="cuda") + offset
    return flat.to(KINDS[kind])[shift:].as_strided((n, dim), (dim + extra, 1))


def params(dim, kind, seed, shift=0):
    w, b = (torch.randn(dim + shift, generator=generator(seed + i), device="cuda").to(KINDS[kind])[shift:] for i in (0, 1))
    return w, b


def host(t):
    return t.detach().double().cpu().numpy()


def chain(dim):
    return max(48, dim / 1024 + 24)


def check_forward(x, w, b, eps, got, kind):
    y, stats = got
    want, right = O.layer_norm(host(x), None if w is None else host(w), None if b is None else host(b), np.float32(eps))
    c = chain(x.shape[-1])
    mean, r = right[..., :1], right[..., 1:]
    off = (c + 1) * U * np.abs(host(x)).mean(-1, keepdims=True)
    assert np.all(np.abs(host(stats)[..., :1] - mean) <= off)
    slack = (c + 8) * U + (off * r) ** 2
    assert np.all(np.abs(host(stats)[..., 1:] - r) <= slack * r)
    scale = 1.0 if w is None else np.abs(host(w))
    xh = np.abs((host(x) - mean) * r) * scale
    bound = scale * r * off * (1 + slack) + xh * (slack + 4 * U) + U * np.abs(want) + U * (0 if b is None else np.abs(host(b))) \
        + HALF[kind] * np.abs(want) * (1 + 2 ** -6)
    assert np.all(np.abs(host(y) - want) <= bound)


@pytest.mark.parametrize("kind,param_kind", [("f32", "f32"), ("bf16", "f32"), ("bf16", "bf16"), ("f32", "bf16")])
@pytest.mark.parametrize("dim", DIMS)
def test_forward(dim, kind, param_kind):
    for n, extra, shift in ((1, 0, 0), (5, 8, 0), (37, 0, 0), (6, 3, 1), (3, 4, 2), (140, 1, 0)):
        x = rows(n, dim, kind, dim, extra, shift)
        w, b = params(dim, param_kind, 7, shift)
        for weight, bias in ((w, b), (w, None), (None, None)):
            wide = torch.full((n, dim + 8), 7.0, dtype=x.dtype, device="cuda")
            got = layer_norm(x, weight, bias, eps=1e-5, out=wide[:, :dim])
            check_forward(x, weight, bias, 1e-5, got, kind)
            assert bool((wide[:, dim:] == 7.0).all())


def check_backward(x, g, stats, w, kind, param_kind, **how):
    n, dim = x.shape
    gw, gb = (torch.full((dim,), 7.0, dtype=KINDS[param_kind], device="cuda") for _ in (0, 1))
    wide = torch.full((n, dim + 8), 7.0, dtype=x.dtype, device="cuda")
    dx, dw, db = layer_norm_backward(g, x, stats, w, gw, gb, out=wide[:, :dim], **how)
    assert dw is gw and db is gb and bool((wide[:, dim:] == 7.0).all())
    want, want_w, want_b = O.layer_norm_backward(host(g), host(x), host(stats), None if w is None else host(w))
    c = chain(dim)
    r = np.abs(host(stats)[:, 1:])
    xh = np.abs((host(x) - host(stats)[:, :1]) * r)
    gg = np.abs(host(g)) * (1.0 if w is None else np.abs(host(w)))
    bound = r * (c + 12) * U * (gg + gg.mean(1, keepdims=True) + xh * (gg * xh).mean(1, keepdims=True)) + HALF[kind] * np.abs(want)
    assert np.all(np.abs(host(dx) - want) <= bound)
    for got, right, terms in ((dw, want_w, np.abs(host(g)) * xh), (db, want_b, np.abs(host(g)))):
        assert np.all(np.abs(host(got) - right) <= (n + 80) * U * terms.sum(0) + HALF[param_kind] * np.abs(right) * (1 + 2 ** -6))
    return dx, dw, db


@pytest.mark.parametrize("kind,param_kind", [("f32", "f32"), ("bf16", "f32"), ("bf16", "bf16"), ("f32", "bf16")])
@pytest.mark.parametrize("dim", DIMS)
def test_backward(dim, kind, param_kind):
    for n, extra, shift in ((1, 0, 0), (5, 8, 0), (131, 0, 0), (6, 3, 1), (3, 4, 2), (140, 1, 0)):
        x, g = rows(n, dim, kind, dim, extra, shift), rows(n, dim, kind, dim + 1, extra, shift, 0.1)
        w, _ = params(dim, param_kind, 7, shift)
        stats = layer_norm(x, w)[1]
        for weight in (w, None):
            full = check_backward(x, g, stats, weight, kind, param_kind)
        # parts of the answer are the same bits as the whole
        gw = torch.empty_like(full[1])
        assert torch.equal(layer_norm_backward(g, x, stats, weight, grad_weight=gw, input_grad=False)[1], full[1])
        assert torch.equal(layer_norm_backward(g, x, stats, weight)[0], full[0])


@pytest.mark.parametrize("n,dim", [(5000, 64), (3000, 264), (7001, 8), (2000, 1024), (40000, 16)])
def test_many_rows(n, dim):
    x, g = rows(n, dim, "bf16", 1), rows(n, dim, "bf16", 2, offset=0.0)
    w, b = params(dim, "f32", 3)
    got = layer_norm(x, w, b)
    check_forward(x, w, b, 1e-5, got, "bf16")
    dx, dw, db = check_backward(x, g, got[1], w, "bf16", "f32")
    again = layer_norm_backward(g, x, got[1], w, torch.empty_like(dw), torch.empty_like(db))
    assert all(torch.equal(a, c) for a, c in zip(again, (dx, dw, db)))        # the same bits
    field_w, field_b = torch.ones_like(dw), torch.full_like(db, 2.0)
    layer_norm_backward(g, x, got[1], w, field_w, field_b, accumulate=True)
    assert torch.equal(field_w, 1 + dw) and torch.equal(field_b, 2 + db)


def test_rows_far_from_zero():
    """A variance about the mean, not a difference of sums: values of 1000 and a spread of 1."""
    for dim in (64, 256, 1024, 4096, 40000):
        x = rows(4, dim, "f32", 5, offset=1000.0)
        check_forward(x, None, None, 1e-5, layer_norm(x), "f32")


def test_constant_rows_and_values_that_are_not_finite():
    for dim in (7, 512, 1000, 5000, 40000):
        x = torch.full((4, dim), 3.0, device="cuda")
        x[1, dim // 2] = float("nan")
        x[2, 0] = float("inf")
        w, b = params(dim, "f32", 1)
        y, stats = layer_norm(x, w, b)
        assert torch.equal(y[0], b) and torch.equal(y[3], b)
        assert bool(torch.isnan(y[1]).all()) and bool(torch.isnan(y[2]).any())
        dx, dw, db = layer_norm_backward(torch.ones_like(x), x, stats, w, torch.empty_like(w), torch.empty_like(w))
        assert bool(torch.isfinite(dx[0]).all()) and bool(torch.isnan(dx[1]).all()) and bool(torch.isfinite(db).all())


def test_no_rows():
    x, w = torch.empty(0, 16, device="cuda"), torch.ones(16, device="cuda")
    y, stats = layer_norm(x, w, w)
    assert y.shape == (0, 16) and stats.shape == (0, 2)
    gw, gb = torch.full((16,), 7.0, device="cuda"), torch.full((16,), 7.0, device="cuda")
    layer_norm_backward(x, x, stats, w, gw, gb, accumulate=True)
    assert bool((gw == 7).all())
    layer_norm_backward(x, x, stats, w, gw, gb)
    assert bool((gw == 0).all()) and bool((gb == 0).all())


def test_autograd():
    x = rows(6, 40, "f32", 1).contiguous().view(2, 3, 40).requires_grad_(True)
    w, b = (t.requires_grad_(True) for t in params(40, "f32", 2))
    g = rows(6, 40, "f32", 3).view(2, 3, 40)
    layer_normed(x, w, b).backward(g)
    stats = layer_norm(x.detach(), w.detach(), b.detach())[1].view(6, 2)
    want = layer_norm_backward(g.view(6, 40), x.detach().view(6, 40), stats, w.detach(), torch.empty(40, device="cuda"),
                               torch.empty(40, device="cuda"))
    assert torch.equal(x.grad.view(6, 40), want[0]) and torch.equal(w.grad, want[1]) and torch.equal(b.grad, want[2])
    field = torch.ones(40, device="cuda"), torch.ones(40, device="cuda")
    x.grad = w.grad = b.grad = None
    layer_normed(x, w, b, grad_into=field).backward(g)
    assert w.grad is None and b.grad is None and torch.equal(field[0], 1 + want[1]) and torch.equal(field[1], 1 + want[2])
    # broadcast gradients, and each set of leaves
    for need in ((1, 0, 0), (0, 1, 0), (0, 0, 1), (1, 1, 1)):
        leaves = [t.detach().clone().requires_grad_(bool(n)) for t, n in zip((x, w, b), need)]
        layer_normed(*leaves).sum().backward()
        assert [t.grad is not None for t in leaves] == [bool(n) for n in need]
    assert torch.equal(b.detach() * 0 + 6, leaves[2].grad)
    plain = x.detach().clone().requires_grad_(True)
    layer_normed(plain).sum().backward()
    assert plain.grad.abs().max() < 1e-4


def test_captured_steps():
    x, g = rows(300, 1024, "bf16", 1), rows(300, 1024, "bf16", 2)
    w, b = params(1024, "f32", 3)
    y, stats = layer_norm(x, w, b)
    gw, gb = torch.empty_like(w), torch.empty_like(b)
    want = [t.clone() for t in (y, stats, *layer_norm_backward(g, x, stats, w, gw, gb))]
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        y2, stats2 = layer_norm(x, w, b)
        dx, _, _ = layer_norm_backward(g, x, stats2, w, gw, gb)
    for _ in range(2):
        gw.zero_(), gb.zero_(), y2.zero_(), dx.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, c) for a, c in zip((y2, stats2, dx, gw, gb), want))
