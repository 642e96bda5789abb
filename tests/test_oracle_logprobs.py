"""The fp64 oracle of log-probabilities and distillation, pinned to facts that
hold apart from it: hand-computed values, limits, and central differences."""
import math

import numpy as np
import pytest

from oracle import tp_oracle as O


def test_hand_computed_row():
    # exp(z) = 1, 2, 5 over 8
    x = np.log(np.array([[1.0, 2.0, 5.0]]))
    r = O.logprobs(x, [1], top_k=2)
    assert math.isclose(r["lse"][0], math.log(8))
    assert math.isclose(r["logprob"][0], math.log(0.25))
    want = -(0.125 * math.log(0.125) + 0.25 * math.log(0.25) + 0.625 * math.log(0.625))
    assert math.isclose(r["entropy"][0], want)
    assert r["top_idx"].tolist() == [[2, 1]]
    assert np.allclose(np.exp(r["top_logprob"]), [[0.625, 0.25]])
    # at scale 2 the weights are 1, 4, 25 over 30
    assert math.isclose(O.logprobs(x, [2], 2.0)["logprob"][0], math.log(25 / 30))


def test_limits():
    v = 64
    r = O.logprobs(np.zeros((1, v)), [3], top_k=5)
    assert math.isclose(r["entropy"][0], math.log(v)) and r["top_idx"].tolist() == [[0, 1, 2, 3, 4]]
    one = np.full((1, v), -np.inf)
    one[0, 7] = 3.0
    r = O.logprobs(one, [7], top_k=3)
    assert r["entropy"][0] == 0.0 and r["logprob"][0] == 0.0 and r["top_idx"].tolist() == [[7, 0, 1]]
    assert r["top_logprob"][0, 1] == -np.inf
    none = O.logprobs(np.full((1, v), -np.inf), [0], top_k=1)
    assert none["lse"][0] == -np.inf and np.isnan(none["entropy"][0]) and np.isnan(none["logprob"][0])


def test_agrees_with_the_cross_entropy():
    g = np.random.default_rng(0)
    x, y = g.normal(size=(9, 50)), g.integers(0, 50, 9)
    r, c = O.logprobs(x, y, top_k=1), O.xent(x, y)
    assert np.allclose(-r["logprob"], c["loss"]) and np.allclose(r["lse"], c["lse"])
    assert np.array_equal(r["top_idx"][:, 0], c["argmax"])
    assert np.allclose(-O.logprobs_bwd(x, y, np.ones(9), None), c["dlogits"])
    d = O.distill(x, y[:, None], np.zeros((9, 1)))
    assert np.allclose(d["loss"], c["loss"]) and np.allclose(d["dlogits"], c["dlogits"])


def _differences(f, x, delta=1e-5):
    d = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        a, b = x.copy(), x.copy()
        a[i] += delta
        b[i] -= delta
        d[i] = (f(a) - f(b)) / (2 * delta)
    return d


@pytest.mark.parametrize("scale", [1.0, 0.6])
def test_gradients_against_differences(scale):
    g = np.random.default_rng(1)
    x, y = g.normal(size=(3, 11)), g.integers(0, 11, 3)
    dlp, de = g.normal(size=3), g.normal(size=3)

    def f(a):
        r = O.logprobs(a, y, scale)
        return (dlp * r["logprob"] + de * r["entropy"]).sum()

    assert np.allclose(O.logprobs_bwd(x, y, dlp, de, scale), _differences(f, x), atol=1e-8)
    ids = np.array([[1, 4, 1], [2, -1, 9], [-1, -1, -1]])       # a token twice, an empty slot, none
    t, w = g.normal(size=(3, 3)), np.array([1.0, 0.5, 2.0])
    for renorm in (True, False):
        r = O.distill(x, ids, t, renorm, w, scale, 0.7)
        d = _differences(lambda a: 0.7 * O.distill(a, ids, t, renorm, w, scale)["loss_sum"], x)
        assert np.allclose(r["dlogits"], d, atol=1e-8) and not r["dlogits"][2].any()


def test_distillation_from_itself_is_zero():
    g = np.random.default_rng(2)
    x = g.normal(size=(4, 20))
    lp = x - O.logprobs(x)["lse"][:, None]
    ids = np.argsort(-x, axis=1)
    r = O.distill(x, ids, np.take_along_axis(lp, ids, 1), renormalize=False)
    assert np.abs(r["loss"]).max() < 1e-12 and np.abs(r["dlogits"]).max() < 1e-12
    top = O.distill(x, ids[:, :5], np.take_along_axis(lp, ids, 1)[:, :5])
    assert (top["loss"] > 0).all()
