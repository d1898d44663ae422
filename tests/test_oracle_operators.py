"""What pins the oracle's AdamW, 8-bit moments and routing (no GPU)."""

import numpy as np
import pytest
import torch

from oracle import adamw as A
from oracle import route as R


def test_adamw_equals_torch_in_double_over_steps():
    rng = np.random.default_rng(0)
    w = rng.normal(size=300)
    p = torch.nn.Parameter(torch.tensor(w))
    opt = torch.optim.AdamW([p], lr=3e-3, betas=(0.8, 0.95), eps=1e-6, weight_decay=0.1)
    m, v = np.zeros(300), np.zeros(300)
    for t in range(1, 8):
        g = rng.normal(size=300)
        p.grad = torch.tensor(g)
        opt.step()
        w, m, v = A.adamw(w, g, m, v, t, 3e-3, 0.8, 0.95, 1e-6, 0.1)
        np.testing.assert_allclose(w, p.detach().numpy(), rtol=1e-13, atol=1e-15)


def test_clip_and_norm():
    g = [np.array([3.0, 0.0]), np.array([4.0])]
    assert A.grad_norm(g) == 5.0 and A.grad_norm([]) == 0.0
    assert A.clip_factor(5.0, 1.0) == pytest.approx(0.2, rel=1e-6)
    assert A.clip_factor(0.5, 1.0) == 1.0 and A.clip_factor(5.0, 0.0) == 1.0


@pytest.mark.parametrize("kind,dtype", [(A.E4M3, torch.float8_e4m3fn), (A.E5M2, torch.float8_e5m2)])
def test_encode_gives_neighbouring_numbers_of_the_format(kind, dtype):
    rng = np.random.default_rng(1)
    x = rng.normal(size=1000) * np.exp(rng.normal(size=1000) * 4)
    z, scale, _ = A.encode(x, rng.integers(0, 65536, 1000), **kind)
    assert np.array_equal(torch.tensor(z).to(dtype).double().numpy(), z)      # numbers of the format
    y = x / np.repeat(scale, A.BLOCK)[:1000]
    # the number below or the one above; the format's largest at most
    assert np.all(np.abs(z - y) < A.spacing(np.abs(y), kind["mantissa"], kind["least"]) * (1 + 1e-9))
    assert np.abs(z).max() == kind["top"]


def test_encode_is_unbiased_over_all_random_bits():
    x = np.array([1.0, 0.3, -0.01, 1e-4, 2.5e-6] + [0.0] * 251)
    r = np.arange(65536)
    for i in range(5):
        got = np.zeros(65536)
        scale = 1.0 / 448
        y = abs(x[i]) / scale
        q = A.spacing(np.array([y]), 3, -6)[0]
        got = np.floor(y / q + r / 65536) * q * scale
        assert abs(got.mean() - abs(x[i])) <= q * scale / 65536
        z, s, _ = A.encode(x, np.full(256, 40000), **A.E4M3)
        assert abs(z[i] * s[0]) == pytest.approx(np.floor(y / q + 40000 / 65536) * q * scale, rel=1e-12)


def test_random_bits_are_spread():
    """4096 blocks: every bit's mean, and products of neighbours, within five standard deviations."""
    n = 4096 * 256
    h = A.random_bits(7, np.repeat(np.arange(4096), 256), np.tile(np.arange(256), 4096))
    other = A.random_bits(8, np.repeat(np.arange(4096), 256), np.tile(np.arange(256), 4096))
    for bit in range(32):
        assert abs(((h >> np.uint64(bit)) & np.uint64(1)).mean() - 0.5) < 5 * 0.5 / np.sqrt(n)
    u, w, z = ((x % 65536) / 65536 - 0.5 for x in (h, h >> np.uint64(16), other))
    for a, b in ((u, w), (u[1:], u[:-1]), (u[256:], u[:-256]), (w[1:], w[:-1]), (u, z)):
        assert abs((a * b).mean()) < 5 / 12 / np.sqrt(n)


def test_route_by_hand():
    x = [1.0, 3.0, 3.0, -np.inf, 2.0, 0.0]
    assert R.route_token(x, 3)[0] == [1, 2, 4]                       # the tie to the lower place
    i, w, _ = R.route_token(x, 2, renorm=True, scale=2.0)
    assert i == [1, 2] and np.allclose(w, [1.0, 1.0])
    # the bias chooses, the score weighs
    i, w, _ = R.route_token([0.0, 1.0], 1, score="sigmoid", bias=np.array([1.0, 0.0]))
    assert i == [0] and np.allclose(w, [0.5])
    # groups of two: worth 0.5 + 0.5 against sigmoid(3) + sigmoid(-9)
    i, _, _ = R.route_token([0.0, 0.0, 3.0, -9.0], 1, score="sigmoid", groups=2, top_groups=1)
    assert i == [0]
    i, w, _ = R.route_token([-np.inf, -np.inf, 1.0], 2, renorm=True)
    assert i == [2, -1] and np.allclose(w, [1.0, 0.0])
    assert R.route_token([-np.inf] * 3, 2)[0] == [-1, -1]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_gradient_against_differences(score, renorm):
    rng = np.random.default_rng(3)
    x, g = rng.normal(size=7), rng.normal(size=3)
    index = [5, 0, -1]
    d = R.backward_token(x, index, g, score, renorm, 2.5)
    h = 1e-5
    for i in range(7):
        up, down = x.copy(), x.copy()
        up[i] += h
        down[i] -= h
        diff = (g @ R.weights_at(up, index, score, renorm, 2.5) - g @ R.weights_at(down, index, score, renorm, 2.5)) / (2 * h)
        assert d[i] == pytest.approx(diff, abs=1e-9)
