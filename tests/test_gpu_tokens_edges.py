"""Embedding, layer norm, dropout and token log probabilities where calls are rare: offsets past 32 bits, rows that start
anywhere, two calls at once, captured passes with another stream's memory, vocabularies between the layouts.

Where a call on a part of the rows is compared with the whole's, each row's arithmetic is the same and the bits are."""

import numpy as np
import pytest
import torch

from oracle import tokens as O
from reduction_reducer_gb300 import (drop, dropped, embed, embed_backward, embedded, layer_norm, layer_norm_backward,
                                     layer_normed, logprobs, logprobs_backward, scored)

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
KINDS = {"f32": torch.float32, "bf16": torch.bfloat16}
HALF = {"f32": U, "bf16": 2.0 ** -8}


@pytest.fixture(scope="module", autouse=True)
def _device():
    torch.cuda.set_device(0)
    yield
    torch.cuda.empty_cache()


def generator(seed):
    return torch.Generator("cuda").manual_seed(seed)


def draw(n, dim, kind, seed, extra=0, shift=0):
    """n rows, `extra` elements apart, from `shift` elements behind a 256-byte boundary on."""
    flat = torch.randn(n * (dim + extra) + shift, generator=generator(seed), device="cuda").to(KINDS[kind])
    return flat[shift:].as_strided((n, dim), (dim + extra, 1))


def host(t):
    return t.detach().double().cpu().numpy()


# ---------------------------------------------------------------- offsets past 32 bits

FAR = 1_100_000            # rows of 2,048: 2.25e9 elements


def far_rows():
    x = torch.zeros(FAR, 2048, dtype=torch.bfloat16, device="cuda")
    x[-300:] = draw(300, 2048, "bf16", 1)
    return x


def test_rows_past_32_bits_of_elements():
    x = far_rows()
    last = x[-300:].clone()
    assert x.numel() > 2 ** 31
    y, stats = layer_norm(x)
    want, want_stats = layer_norm(last)
    assert torch.equal(y[-300:], want) and torch.equal(stats[-300:], want_stats)
    grad = y                                               # any
    dx, _, _ = layer_norm_backward(grad, x, stats)
    assert torch.equal(dx[-300:], layer_norm_backward(want, last, want_stats)[0])
    del y, dx, grad
    got = drop(x, 0.25, 7, residual=x)
    keep = np.array([[O.random_bits((FAR - 2) * 2048 + r * 2048 + c, 7, 0) >= 2 ** 30 for c in range(64)] for r in range(2)])
    exact = host(last[-2:, :64]) * (1 + keep / 0.75)
    assert np.all(np.abs(host(got[-2:, :64]) - exact) <= (2.0 ** -8 + 4 * U) * 3 * np.abs(host(last[-2:, :64])))
    del got
    t = torch.randint(2048, (FAR,), generator=generator(2), device="cuda")
    t[:-300] = -1
    full, part = logprobs(x, t, 2, entropy=True), logprobs(last, t[-300:].clone(), 2, entropy=True)
    assert all(torch.equal(a[-300:], b) for a, b in zip(full, part))
    one = torch.ones(FAR, device="cuda")
    d = logprobs_backward(one, x, t, full.stats, out=x)
    assert torch.equal(d[-300:], logprobs_backward(one[:300], last, t[-300:].clone(), part.stats))
    assert not bool(d[:4].any())


def test_tables_past_32_bits_of_elements():
    table = far_rows()
    tokens = torch.tensor([FAR - 1, 0, FAR - 300, FAR - 1, FAR, FAR - 7], device="cuda")
    want = table[tokens.clamp(max=FAR - 1)]
    want[4] = 0
    assert torch.equal(embed(table, tokens), want)
    grad = draw(6, 2048, "bf16", 3)
    embed_backward(grad, tokens, table)
    assert torch.equal(table[FAR - 1], (grad[0].float() + grad[3].float()).bfloat16())
    assert torch.equal(table[FAR - 7], grad[5]) and torch.equal(table[FAR - 300], grad[2]) and torch.equal(table[0], grad[1])
    assert not bool(table[-6:-1].any()) and not bool(table[1:4].any())


def test_gradients_past_32_bits_of_elements():
    grad = far_rows()
    tokens = torch.full((FAR,), -1, device="cuda")
    tokens[-300:] = torch.randint(50, (300,), generator=generator(4), device="cuda")
    got = embed_backward(grad, tokens, torch.empty(50, 2048, device="cuda"))
    want, size, count = O.embed_backward(host(grad[-300:]), tokens[-300:].cpu().numpy(), 50)
    assert np.all(np.abs(host(got) - want) <= (count + 3)[:, None] * U * size)


# ---------------------------------------------------------------- rows that start anywhere

@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("shift,extra", [(0, 4), (4, 0), (4, 8), (8, 4), (1, 0), (2, 6), (3, 3)])
def test_rows_that_start_anywhere(shift, extra, kind):
    n, dim = 37, 264
    x = draw(n, dim, kind, shift, extra, shift)
    flat = x.contiguous()

    def place(like):
        out = torch.full((like.shape[0] * (like.shape[1] + extra) + shift,), 7.0, dtype=like.dtype, device="cuda")
        return out, out[shift:].as_strided(like.shape, (like.shape[1] + extra, 1))

    def check(call, want):
        whole, out = place(want)
        call(out)
        assert torch.equal(out, want)
        out.fill_(7.0)
        assert bool((whole == 7.0).all())                   # nothing between the rows or around them

    check(lambda out: drop(x, 0.3, 5, out=out), drop(flat, 0.3, 5))
    check(lambda out: drop(x, 0.3, 5, residual=x, out=out), drop(flat, 0.3, 5, residual=flat))
    tokens = torch.randint(-1, n + 1, (100,), generator=generator(1), device="cuda")
    check(lambda out: embed(x, tokens, scale=0.7, out=out), embed(flat, tokens, scale=0.7))
    grad = draw(100, dim, kind, 2, extra, shift)
    for table in KINDS.values():
        want = embed_backward(grad.contiguous(), tokens, torch.empty(n, dim, dtype=table, device="cuda"))
        check(lambda out: embed_backward(grad, tokens, out), want)
    check(lambda out: embed_backward(grad, tokens, out.zero_(), accumulate=True) if kind == "f32" else out.copy_(want), want
          if kind == "bf16" else embed_backward(grad.contiguous(), tokens, torch.zeros(n, dim, device="cuda"), accumulate=True))
    # sums over a row are in another order where rows do not lie alike: compared with 64 bits
    y, stats = O.layer_norm(host(x))
    whole, out = place(flat)
    got, got_stats = layer_norm(x, out=out)
    assert np.all(np.abs(host(got) - y) <= HALF[kind] * np.abs(y) + 600 * U * (1 + np.abs(y)))
    t = torch.randint(dim, (n,), generator=generator(3), device="cuda")
    scores = logprobs(x, t, 4, entropy=True)
    alike = logprobs(flat, t, 4, entropy=True)
    assert torch.equal(scores.top_index, alike.top_index)
    # 264 terms of at most 1 in the sum, each within 8 u
    assert torch.allclose(scores.logp, alike.logp, rtol=0, atol=2 * 272 * U * 8)
    check(lambda out: logprobs_backward(t.float(), x, t, scores.stats, out=out), logprobs_backward(t.float(), flat, t, scores.stats))


# ---------------------------------------------------------------- vocabularies between the layouts

@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("n,vocab,top", [(1215, 8192, 0), (1216, 8192, 0), (1217, 8193, 0), (2431, 5120, 6), (2432, 5120, 32),
                                         (2433, 5121, 1), (2433, 2049, 7), (911, 8192, 3), (912, 8192, 3),
                                         (2432, 16384, 20), (2431, 16384, 20)])
def test_many_rows_of_middling_vocabularies(n, vocab, top, kind):
    """Against single rows, which have eight warps each; sums of fewer than 2^13 terms that are at most 1, of the largest
    being 1: their order and the exponentials' errors come to less than 2^9 u (for sums by lanes of 2^13 / 32 terms)."""
    x = draw(n, vocab, kind, 1, shift=1)
    t = torch.randint(-1, vocab, (n,), generator=generator(2), device="cuda")
    got = logprobs(x, t, top, 0.9, entropy=True)
    d = logprobs_backward(torch.ones(n, device="cuda"), x, t, got.stats, 0.9)
    for i in (0, 7, 8, n // 2, n - 2, n - 1):
        one = logprobs(x[i:i + 1], t[i:i + 1], top, 0.9, entropy=True)
        if top:
            assert torch.equal(one.top_index[0], got.top_index[i])
            assert torch.allclose(one.top_logp[0], got.top_logp[i], rtol=0, atol=600 * U)
        assert torch.allclose(one.logp[0], got.logp[i], rtol=0, atol=600 * U)
        assert torch.allclose(one.entropy[0], got.entropy[i], rtol=0, atol=6000 * U)
        if int(t[i]) >= 0:
            p = torch.softmax(x[i].double() * 0.9, 0)
            want = 0.9 * (torch.nn.functional.one_hot(t[i], vocab).double() - p)
            assert bool(((d[i].double() - want).abs() <= HALF[kind] * want.abs() + 700 * U * p).all())
        else:
            assert not bool(d[i].any()) and float(got.logp[i]) == 0.0


# ---------------------------------------------------------------- streams and graphs

def model(table, w, b, tokens, targets, seed):
    x = dropped(embedded(table, tokens, 3.0), 0.2, seed)
    y = layer_normed(x, w, b)
    x = dropped(y, 0.2, seed, 1, residual=x)
    return scored(x @ table.t(), targets, entropy=True)


def test_two_calls_at_once():
    """Each call's workspace is its own: two streams at a time give what they give one after another."""
    grads = [draw(20000, 72, "bf16", i) for i in range(2)]
    tokens = [torch.randint(30, (20000,), generator=generator(i), device="cuda") for i in range(2)]
    x, w = [g.contiguous() for g in grads], torch.ones(72, device="cuda")

    def both(streams):
        torch.cuda.synchronize()
        out = []
        for _ in range(5):
            for g, t, s in zip(grads, tokens, streams):
                with torch.cuda.stream(s):
                    table = embed_backward(g, t, torch.empty(30, 72, device="cuda"))
                    y, stats = layer_norm(g, w, w)
                    gw, gb = torch.empty(72, device="cuda"), torch.empty(72, device="cuda")
                    dx, _, _ = layer_norm_backward(y, g, stats, w, gw, gb)
                    out += [table, y, dx, gw, gb]
        torch.cuda.synchronize()
        return out

    main = torch.cuda.current_stream()
    want = both((main, main))
    got = both((torch.cuda.Stream(), torch.cuda.Stream()))
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    assert len(x) == 2


def test_workspaces_of_the_caller():
    grad, tokens = draw(3000, 40, "f32", 1), torch.randint(50, (3000,), generator=generator(1), device="cuda")
    want = embed_backward(grad, tokens, torch.empty(50, 40, device="cuda"))
    space = torch.full((1 << 24,), 255, dtype=torch.uint8, device="cuda")       # what it holds does not matter
    for _ in range(2):
        assert torch.equal(embed_backward(grad, tokens, torch.empty(50, 40, device="cuda"), workspace=space), want)
    y, stats = layer_norm(grad)
    sums = [torch.empty(40, device="cuda") for _ in range(4)]
    layer_norm_backward(y, grad, stats, None, sums[0], sums[1])
    layer_norm_backward(y, grad, stats, None, sums[2], sums[3], workspace=space)
    assert torch.equal(sums[0], sums[2]) and torch.equal(sums[1], sums[3])
    with pytest.raises(ValueError, match="workspace"):
        embed_backward(grad, tokens, torch.empty(50, 40, device="cuda"), workspace=space[:100])
    with pytest.raises(ValueError, match="workspace"):
        layer_norm_backward(y, grad, stats, None, sums[0], sums[1], workspace=space[:100])


def test_captured_training_passes():
    """Two graphs of whole passes, replayed in turn with new tokens and a new seed each time."""
    table = draw(97, 64, "f32", 1).contiguous().requires_grad_(True)
    w, b = torch.ones(64, device="cuda", requires_grad=True), torch.zeros(64, device="cuda", requires_grad=True)
    tokens = torch.zeros(2, 50, dtype=torch.int64, device="cuda")
    targets, seed = torch.zeros_like(tokens), torch.zeros(1, dtype=torch.int64, device="cuda")

    def step(scale):
        got = model(table, w, b, tokens, targets, seed)
        loss = -(got.logp.sum() + 0.1 * got.entropy.sum()) * scale
        return (loss.detach(), *torch.autograd.grad(loss, (table, w, b)))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(1.0)
    torch.cuda.current_stream().wait_stream(side)
    graphs, held = [torch.cuda.CUDAGraph() for _ in range(2)], []
    for i, g in enumerate(graphs):
        with torch.cuda.graph(g):
            held.append(step(1.0 + i))
    for turn in range(3):
        tokens.copy_(torch.randint(-1, 97, (2, 50), generator=generator(turn), device="cuda"))
        targets.copy_(torch.randint(-1, 97, (2, 50), generator=generator(turn + 9), device="cuda"))
        seed.fill_(turn)
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for i in range(2):
            want = step(1.0 + i)
            assert all(torch.allclose(a, b, rtol=1e-5, atol=1e-5) for a, b in zip(held[i], want))
            # what no library product has a part in is the same bit for bit
            assert torch.equal(held[i][0], want[0])


# ---------------------------------------------------------------- refusals

def test_fields_of_parameters_that_are_not_fp32_are_refused():
    x, w = draw(4, 16, "bf16", 1).contiguous(), torch.ones(16, dtype=torch.bfloat16, device="cuda", requires_grad=True)
    with pytest.raises(ValueError, match="grad_into"):
        layer_normed(x, w, None, grad_into=(torch.zeros(16, device="cuda"), None))
    table = draw(9, 16, "bf16", 1).contiguous().requires_grad_(True)
    with pytest.raises(ValueError, match="grad_into"):
        embedded(table, torch.zeros(3, dtype=torch.int64, device="cuda"), grad_into=torch.zeros(9, 16, device="cuda").bfloat16())
    field = torch.zeros(9, 16, device="cuda")              # a bf16 table's gradient in fp32
    embedded(table, torch.zeros(3, dtype=torch.int64, device="cuda"), grad_into=field).float().sum().backward()
    assert bool((field[0] == 3).all()) and not bool(field[1:].any())
