"""The token operators' oracle: published vectors, closed forms and differences."""

import numpy as np
import pytest

from oracle import tokens as O


@pytest.mark.parametrize("counter,key,words", [
    ((0, 0, 0, 0), (0, 0), (0x6627e8d5, 0xe169c58d, 0xbc57ac4c, 0x9b00dbd8)),
    ((0xffffffff,) * 4, (0xffffffff,) * 2, (0x408f276d, 0x41c83b0e, 0xa20bc7c6, 0x6d5451fd)),
    ((0x243f6a88, 0x85a308d3, 0x13198a2e, 0x03707344), (0xa4093822, 0x299f31d0),
     (0xd16cfe09, 0x94fdcceb, 0x5001e420, 0x24126ea1))])
def test_philox_known_answers(counter, key, words):
    """The known answers that were published with the generator."""
    assert tuple(O.philox(counter, key)) == words


def test_dropout():
    x = np.ones(4000)
    y = O.drop(x, 0.25, 7, 3)
    assert set(np.unique(y)) == {0.0, 4 / 3}
    assert abs((y > 0).mean() - 0.75) < 5 * np.sqrt(0.25 * 0.75 / 4000)
    assert not np.array_equal(y, O.drop(x, 0.25, 7, 4)) and not np.array_equal(y, O.drop(x, 0.25, 8, 3))
    assert np.array_equal(O.drop(x, 0.0, 7), x) and not O.drop(x * np.nan, 1.0, 7).any()


def difference(f, x, by, step=1e-6):
    d = np.zeros_like(x)
    for i in np.ndindex(*x.shape):
        hi, lo = x.copy(), x.copy()
        hi[i] += step
        lo[i] -= step
        d[i] = ((f(hi) - f(lo)) * by).sum() / (2 * step)
    return d


def test_layer_norm_gradients_against_differences():
    rng = np.random.default_rng(0)
    x, w, b, g = rng.normal(size=(3, 5)) + 1, rng.normal(size=5), rng.normal(size=5), rng.normal(size=(3, 5))
    stats = O.layer_norm(x, w, b)[1]
    dx, dw, db = O.layer_norm_backward(g, x, stats, w)
    np.testing.assert_allclose(dx, difference(lambda v: O.layer_norm(v, w, b)[0], x, g), atol=1e-7)
    np.testing.assert_allclose(dw, difference(lambda v: O.layer_norm(x, v, b)[0], w, g), atol=1e-7)
    np.testing.assert_allclose(db, difference(lambda v: O.layer_norm(x, w, v)[0], b, g), atol=1e-7)


def test_embedding_gradient_against_differences():
    rng = np.random.default_rng(1)
    table, tokens, g = rng.normal(size=(4, 3)), np.array([1, 3, 1, -1, 9, 0]), rng.normal(size=(6, 3))
    d, _, count = O.embed_backward(g, tokens, 4, 2.0)
    assert count.tolist() == [1, 2, 0, 1]
    np.testing.assert_allclose(d, difference(lambda t: O.embed(t, tokens, 2.0), table, g), atol=1e-8)


@pytest.mark.parametrize("target", [0, 2, None, 7])
def test_logprob_gradients_against_differences(target):
    x = np.array([0.3, -1.2, 2.0, 0.3, -np.inf])
    live = x > -np.inf

    def both(v):
        logp, entropy, *_ = O.logprobs(np.append(v, -np.inf), target, 0, 0.7)
        return 0.6 * (logp or 0.0) - 0.4 * entropy

    d = O.logprobs_backward(x, target, 0.6, -0.4, 0.7)
    assert d[~live] == 0
    np.testing.assert_allclose(d[live], difference(lambda v: np.array(both(v)), x[live], 1.0), atol=1e-8)


def test_rows_that_leave_nothing():
    inf = np.inf
    assert O.logprobs([-inf, -inf], 0, 1) == (-inf, 0.0, (-inf, 0.0), [-1], [-inf])
    assert O.logprobs([1.0, 2.0], -1, 1) == (0.0, 0.0, (0.0, 0.0), [-1], [0.0])
    logp, entropy, _, index, _ = O.logprobs([1.0, inf], 0, 2)
    assert np.isnan(logp) and np.isnan(entropy) and index == [1, 0]
    assert O.logprobs([3.0, 3.0, 1.0], 0, 3)[3] == [0, 1, 2]
    assert O.logprobs([0.0] * 4, 1)[1] == pytest.approx(np.log(4))
