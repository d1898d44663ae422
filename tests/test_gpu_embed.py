"""Embedding and its gradient on the GPU against the 64-bit oracle.

Bounds (u = 2^-24, h = half a step of the result's type): a row is one fp32
product and one rounding, u + h of its value.  A row of the gradient adds n terms
one after another (in parts, which only shortens chains): n u of the sum of
their magnitudes, and u each for scale, the sum with what was there, and h."""

import numpy as np
import pytest
import torch

from oracle import tokens as O
from reduction_reducer_gb300 import embed, embed_backward, embedded

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
KINDS = {"f32": torch.float32, "bf16": torch.bfloat16}
HALF = {"f32": U, "bf16": 2.0 ** -8}


@pytest.fixture(scope="module", autouse=True)
def _device():
    torch.cuda.set_device(0)


def generator(seed):
    return torch.Generator("cuda").manual_seed(seed)


def rows(n, dim, kind, seed, extra=0, shift=0):
    """n rows, `extra` elements apart, from `shift` elements behind a 16-byte boundary on."""
    flat = torch.randn(max(n, 1) * (dim + extra) + shift, generator=generator(seed), device="cuda").to(KINDS[kind])
    return flat[shift:].as_strided((n, dim), (dim + extra, 1))


def words(n, vocab, seed, outside=True):
    t = (torch.rand(n, generator=generator(seed), device="cuda") ** 3 * vocab).long()
    if outside:
        t[::7], t[3::11] = -1, vocab
    return t


def host(t):
    return t.detach().double().cpu().numpy()


SHAPES = [(1, 5, 8), (7, 3, 1), (33, 50, 24), (5, 11, 769), (300, 40, 64), (130, 1000, 256), (64, 20, 1000), (9, 7, 2056)]


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("table_kind", ["f32", "bf16"])
@pytest.mark.parametrize("n,vocab,dim", SHAPES)
def test_embed(n, vocab, dim, table_kind, kind):
    for bits, extra, shift in ((torch.int32, 0, 0), (torch.int64, 8, 0), (torch.int64, 3, 1)):
        table = rows(vocab, dim, table_kind, 1, extra, shift)
        tokens = words(n, vocab, 2).to(bits)
        wide = torch.full((n, dim + 8), 7.0, dtype=KINDS[kind], device="cuda")
        got = embed(table, tokens, scale=1.7, out=wide[:, :dim])
        assert bool((wide[:, dim:] == 7.0).all())
        want = O.embed(host(table), tokens.cpu().numpy(), np.float32(1.7))
        assert np.all(np.abs(host(got) - want) <= (U + HALF[kind]) * np.abs(want))
        assert torch.equal(embed(table, tokens, scale=1.7, dtype=KINDS[kind]), got)


def check(grad, tokens, vocab, kind, scale, onto=None, out=None, **how):
    fresh = torch.full((vocab, grad.shape[-1]), 7.0, dtype=KINDS[kind], device="cuda") if out is None else out
    if onto is not None:
        fresh.copy_(onto)
    got = embed_backward(grad, tokens, fresh, scale=scale, accumulate=onto is not None, **how)
    assert got is fresh
    want, size, count = O.embed_backward(host(grad), tokens.cpu().numpy(), vocab, float(np.float32(scale)),
                                         None if onto is None else host(onto))
    bound = (count + 3)[:, None] * U * size + HALF[kind] * np.abs(want)
    assert np.all(np.abs(host(got) - want) <= bound)
    assert bool((host(got)[count == 0] == (0 if onto is None else host(onto)[count == 0])).all())
    return got


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("table_kind", ["f32", "bf16"])
@pytest.mark.parametrize("n,vocab,dim", SHAPES)
def test_gradient(n, vocab, dim, table_kind, kind):
    for bits, extra, shift in ((torch.int32, 0, 0), (torch.int64, 8, 0), (torch.int64, 3, 1)):
        grad, tokens = rows(n, dim, kind, 3, extra, shift), words(n, vocab, 4).to(bits)
        first = check(grad, tokens, vocab, table_kind, 0.7)
        wide = torch.full((vocab, dim + 8), 7.0, dtype=KINDS[table_kind], device="cuda")
        assert torch.equal(check(grad, tokens, vocab, table_kind, 0.7, out=wide[:, :dim]), first)
        assert bool((wide[:, dim:] == 7.0).all())
        if table_kind == "f32":
            check(grad, tokens, vocab, table_kind, 0.7, onto=rows(vocab, dim, "f32", 5))


@pytest.mark.parametrize("dim", [8, 40, 7])
@pytest.mark.parametrize("n,vocab,few", [(65, 9, 1), (128, 70000, 1), (129, 2, 1), (1000, 300, 2), (5000, 50000, 3),
                                         (40000, 200, 1), (70000, 70, 4), (3000, 2 ** 24 // 64, 3000)])
def test_tokens_that_fall_often(n, vocab, few, dim):
    """A few words among all others: rows of more tokens than one part, at borders of parts and windows."""
    gen = generator(n)
    chosen = torch.randint(vocab, (few,), generator=gen, device="cuda")
    tokens = torch.where(torch.rand(n, generator=gen, device="cuda") < 0.6,
                         chosen[torch.randint(few, (n,), generator=gen, device="cuda")],
                         torch.randint(vocab, (n,), generator=gen, device="cuda"))
    grad = rows(n, dim, "bf16", 6)
    got = torch.full((vocab, dim), 7.0, device="cuda")
    embed_backward(grad, tokens, got)
    again = torch.full((vocab, dim), 7.0, device="cuda")
    assert torch.equal(embed_backward(grad, tokens, again), got)              # the same bits
    count = torch.bincount(tokens, minlength=vocab)
    want = torch.zeros(vocab, dim, dtype=torch.float64, device="cuda").index_add_(0, tokens, grad.double())
    size = torch.zeros(vocab, dim, dtype=torch.float64, device="cuda").index_add_(0, tokens, grad.double().abs())
    assert bool(((got.double() - want).abs() <= (count + 3).unsqueeze(1) * U * size).all())


@pytest.mark.parametrize("edge", [31, 32, 33, 63, 64, 65, 127, 128, 129, 192, 1023, 1024, 1025, 1056, 1057])
def test_rows_at_the_borders_of_parts(edge):
    """Runs of one token of every length around a part's, after every start."""
    for before in (0, 1, 30, 31, 32, 33, 62, 63, 64, 65):
        tokens = torch.cat([torch.arange(before) % 3, torch.full((edge,), 5), torch.full((70,), 6), torch.full((3,), -1)]).cuda()
        grad = torch.randint(-8, 9, (len(tokens), 16), generator=generator(edge), device="cuda").float()
        want = torch.zeros(9, 16, device="cuda").index_add_(0, tokens.clamp(min=0), grad * (tokens >= 0).unsqueeze(1))
        out = torch.full((9, 16), 7.0, device="cuda")
        assert torch.equal(embed_backward(grad, tokens, out), want)           # whole numbers: sums are exact
        onto = torch.ones(9, 16, device="cuda")
        assert torch.equal(embed_backward(grad, tokens, onto, accumulate=True), want + 1)


def test_a_row_does_not_depend_on_other_tokens():
    grad, tokens = rows(700, 32, "f32", 8), words(700, 40, 9, outside=False)
    all_ = embed_backward(grad, tokens, torch.empty(40, 32, device="cuda"))
    for v in tokens.unique()[:5]:
        mine = tokens == v
        alone = embed_backward(grad[mine], tokens[mine], torch.empty(40, 32, device="cuda"))
        assert torch.equal(alone[v], all_[v])


def test_no_tokens_and_none_in_the_table():
    out = torch.full((5, 16), 7.0, device="cuda")
    none = torch.empty(0, dtype=torch.int64, device="cuda")
    assert embed(out, none).shape == (0, 16)
    embed_backward(torch.empty(0, 16, device="cuda"), none, out, accumulate=True)
    assert bool((out == 7.0).all())
    embed_backward(torch.empty(0, 16, device="cuda"), none, out)
    assert bool((out == 0).all())
    far = torch.tensor([-1, 5, 2 ** 40, -2 ** 40 + 1, 2 ** 32 + 1], device="cuda")
    out.fill_(7.0)
    assert bool((embed(torch.ones(5, 16, device="cuda"), far) == 0).all())
    embed_backward(torch.full((5, 16), float("nan"), device="cuda"), far, out)
    assert bool((out == 0).all())


def test_autograd():
    table = rows(30, 24, "f32", 1).contiguous().requires_grad_(True)
    tokens = words(20, 30, 2).view(4, 5)
    y = embedded(table, tokens, 2.0)
    g = rows(20, 24, "f32", 3).view(4, 5, 24)
    y.backward(g)
    want, size, count = O.embed_backward(host(g), tokens.cpu().numpy(), 30, 2.0)
    assert np.all(np.abs(host(table.grad) - want) <= (count + 3)[:, None] * U * size)
    # into a gradient field, on top of what is there; broadcast gradients; nothing for the table itself
    field, table.grad = torch.ones(30, 24, device="cuda"), None
    embedded(table, tokens, 2.0, grad_into=field).sum().backward()
    assert table.grad is None
    want, size, count = O.embed_backward(np.ones((20, 24)), tokens.cpu().numpy(), 30, 2.0, np.ones((30, 24)))
    assert np.array_equal(host(field), want)
    half = table.detach().bfloat16().requires_grad_(True)
    embedded(half, tokens, dtype=torch.float32).sum().backward()
    assert half.grad.dtype is torch.bfloat16 and half.grad.sum() == (tokens >= 0).logical_and(tokens < 30).sum() * 24
    with pytest.raises(RuntimeError):
        torch.autograd.grad(torch.autograd.grad(embedded(table, tokens).square().sum(), table, create_graph=True)[0].sum(), table)


def test_streams_graphs_and_workspaces():
    grad, tokens = rows(500, 64, "f32", 11), words(500, 90, 12)
    want = embed_backward(grad, tokens, torch.empty(90, 64, device="cuda"))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = torch.empty(90, 64, device="cuda")
    embed_backward(grad, tokens, out, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(out, want)
    graphs, outs, ins = [], [], []
    for i in range(2):                                 # two graphs, each with a workspace of its own
        g, o, x = torch.cuda.CUDAGraph(), torch.zeros(90, 64, device="cuda"), grad * (i + 1)
        torch.cuda.synchronize()
        with torch.cuda.graph(g):
            embed_backward(x, tokens, o)
        graphs.append(g), outs.append(o), ins.append(x)
    for _ in range(3):
        for g, s in zip(graphs, (torch.cuda.current_stream(), side)):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], want)
        assert torch.equal(outs[1], embed_backward(ins[1], tokens, torch.empty(90, 64, device="cuda")))
        [o.zero_() for o in outs]
        torch.cuda.synchronize()


@pytest.mark.parametrize("vocab", [2, 255, 256, 70000])
@pytest.mark.parametrize("n", [1, 31, 1024, 1025, 8191, 8192, 8193, 20000])
def test_both_sorts(n, vocab):
    """Whole numbers around the sizes at which one CTA sorts, and around those of its rounds and digits."""
    tokens = words(n, vocab, n + vocab)
    grad = torch.randint(-4, 5, (n, 16), generator=generator(n), device="cuda").float()
    there = (tokens >= 0) & (tokens < vocab)
    want = torch.zeros(vocab, 16, device="cuda").index_add_(0, tokens.clamp(0, vocab - 1), grad * there.unsqueeze(1))
    out = torch.full((vocab, 16), 7.0, device="cuda")
    assert torch.equal(embed_backward(grad, tokens, out), want)
