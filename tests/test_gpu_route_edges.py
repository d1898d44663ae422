"""Edges of routing and its gradient on the GPU: confident experts, scales near fp32's least, softmax scores by their
definition whatever the batch, and every store path of the gradient."""

import numpy as np
import pytest
import torch

from oracle import route as R
from reduction_reducer_gb300 import route, route_backward

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
KINDS = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _device():
    torch.cuda.set_device(0)


def generator(seed):
    return torch.Generator("cuda").manual_seed(seed)

@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("renorm", [False, True])
def test_sigmoid_gradient_of_confident_experts(renorm, dtype):
    """Chosen logits of 8 to 20, where 1 - s is 3e-4 to 2e-9: its own relative error stays a few roundings (expf 4u, a
    sum and a quotient), those of the weights 64u, so as they are a gradient is within 80u of itself; renormalised it is
    a difference of terms of at most the row's sum of |g w|, which the factor 1 - s multiplies whole."""
    T, E, k, scale = 400, 32, 8, 2.5
    x = (torch.rand(T, E, generator=generator(1), device="cuda") * 12 + 8).to(KINDS[dtype])
    g = torch.randn(T, k, generator=generator(2), device="cuda")
    index, w = route(x, k, score="sigmoid", renorm=renorm, scale=scale)
    d = route_backward(g, x, index, w, score="sigmoid", renorm=renorm, scale=scale).double()
    at = index.long()
    z, gd = x.double().gather(1, at), g.double()
    s, rest = 1 / (1 + torch.exp(-z)), 1 / (1 + torch.exp(z))        # rest: 1 - s without a difference
    if renorm:
        share = s / s.sum(1, keepdim=True)
        want = scale * share * (gd - (gd * share).sum(1, keepdim=True)) * rest
        bound = 160 * U * (gd * share * scale).abs().sum(1, keepdim=True) * rest
    else:
        want = scale * gd * s * rest
        bound = 80 * U * want.abs()
    if dtype == "bf16":
        bound = bound + 2.0 ** -8 * want.abs()
    got = d.gather(1, at)
    assert bool(((got - want).abs() <= bound).all())
    assert int((d != 0).sum()) <= T * k

@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("scale", [1e-39, -3e-40])
def test_gradient_at_scales_below_the_least_normal_number(scale, score):
    """1 / scale is infinite in fp32.  Weights and products are subnormal, each within 2^-150 of itself: k + 4 of these
    beside the bound of ordinary scales."""
    T, E, k = 50, 24, 6
    x = torch.randn(T, E, generator=generator(3), device="cuda")
    g = torch.randn(T, k, generator=generator(4), device="cuda")
    index, w = route(x, k, score=score, renorm=True, scale=scale)
    assert bool((w != 0).all())
    d = route_backward(g, x, index, w, score=score, renorm=True, scale=scale).double().cpu().numpy()
    fp32_scale = float(np.float32(scale))
    for t in range(T):
        gt = g[t].double().cpu().numpy()
        want = R.backward_token(x[t].double().cpu().numpy(), index[t].tolist(), gt, score, True, fp32_scale)
        size = np.abs(gt * w[t].double().cpu().numpy()).sum()
        assert np.all(np.abs(d[t] - want) <= 160 * U * size + (k + 4) * 2.0 ** -149 * (1 + np.abs(gt).max())), t
