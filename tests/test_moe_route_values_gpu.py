"""GPU tests of tq2_moe_route on scores that are not finite or whose probabilities leave f64's range.

Scores are given one by one: x's first column is 1 and the weights hold a score there, exact in any order of summation."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")
TOL = 2.0 ** -23.9               # one rounding to f32 beside the f64 steps


@pytest.fixture(scope="module")
def moe():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a ROCm device")
    from gemv_tq2_g128_amd import moe as mod
    return mod


def run(moe, tokens, scores, top_k, bias=None, **over):
    """Every token has these scores."""
    w = torch.zeros(len(scores), 64)
    w[:, 0] = torch.tensor(scores)
    x = torch.zeros(tokens, 64)
    x[:, 0] = 1.0
    weights, ids = moe.route(x.cuda(), w.cuda(), top_k, bias=None if bias is None else bias.cuda(), **over)
    torch.cuda.synchronize()
    weights, ids = weights.cpu().numpy().astype(np.float64), ids.cpu().numpy()
    assert (ids == ids[0]).all() and np.array_equal(weights, np.repeat(weights[:1], tokens, 0), equal_nan=True)
    return weights[0], ids[0]


def order(by):
    """Experts by falling `by`, the lowest index first among equals, NaN last."""
    return np.argsort(np.where(np.isnan(by), np.inf, -by), kind="stable")


@pytest.mark.parametrize("tokens", [1, 20])
@pytest.mark.parametrize("experts", [40, 300])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [True, False])
def test_nan_scores_come_last_with_a_bias_too(moe, tokens, experts, scoring, renormalize):
    rng = np.random.default_rng(1)
    scores = rng.standard_normal(experts).astype(np.float32)
    scores[[0, 7]] = NAN
    bias = torch.from_numpy(rng.uniform(-0.02, 0.02, experts).astype(np.float32))
    bias[0] = 100.0
    weights, ids = run(moe, tokens, scores, 8, bias, scoring=scoring, renormalize=renormalize)
    e = np.exp(scores.astype(np.float64))
    p = e / np.nansum(e) if scoring == "softmax" else 1 / (1 + 1 / e)
    at = order(p + bias.double().numpy())[:8]
    assert ids.tolist() == at.tolist()
    if scoring == "softmax":
        assert np.isnan(weights).all()
    else:
        want = p[at] / (p[at].sum() if renormalize else 1)
        assert np.abs(weights / want - 1).max() <= TOL
    # Nothing else is left: the NaN ones, by index; one of them makes the sum NaN.
    scores[:] = NAN
    scores[[5, 9]] = 1.0, 2.0
    weights, ids = run(moe, tokens, scores, 4, torch.zeros(experts), scoring=scoring, renormalize=renormalize)
    assert ids.tolist() == [9, 5, 0, 1] and np.isnan(weights[2:]).all()
    assert np.isnan(weights).all() or (scoring == "sigmoid" and not renormalize)
    scores[:] = NAN
    weights, ids = run(moe, tokens, scores, 4, torch.zeros(experts), scoring=scoring, renormalize=renormalize)
    assert ids.tolist() == [0, 1, 2, 3] and np.isnan(weights).all()


@pytest.mark.parametrize("tokens", [1, 20])
def test_infinite_scores_with_a_bias(moe, tokens):
    scores = np.linspace(-1, 1, 70).astype(np.float32)
    scores[[30, 60]] = INF
    scores[3] = NAN
    bias = torch.arange(70).float() * 1e-3
    bias[50] = 0.9
    for given in (bias, -bias):
        p = np.where(np.isnan(scores), NAN, (scores == INF) / 2)
        weights, ids = run(moe, tokens, scores, 6, given)
        assert ids.tolist() == order(p + given.double().numpy())[:6].tolist() and np.isnan(weights).all()
        s = np.where(scores == INF, scores, -INF).astype(np.float32)
        weights, ids = run(moe, tokens, s, 6, given)
        assert ids.tolist() == order((s == INF) / 2 + given.double().numpy())[:6].tolist() and np.isnan(weights).all()
        s[:] = -INF
        weights, ids = run(moe, tokens, s, 6, given)
        assert ids.tolist() == order(1 / 70 + given.double().numpy())[:6].tolist() and np.isnan(weights).all()
        # sigmoid has its limits: 1 and 0.
        s = np.where(scores == INF, scores, -INF).astype(np.float32)
        weights, ids = run(moe, tokens, s, 6, given, scoring="sigmoid", renormalize=False)
        at = order((s == INF) * 1.0 + given.double().numpy())[:6]
        assert ids.tolist() == at.tolist() and np.array_equal(weights, (s[at] == INF) * 1.0)


def shares(scores, at):
    """exp(score) of the chosen by their sum, in extended precision."""
    e = np.exp(scores[at].astype(np.longdouble) - scores[at].astype(np.longdouble).max())
    return (e / e.sum()).astype(np.float64)


@pytest.mark.parametrize("tokens", [1, 20])
@pytest.mark.parametrize("experts", [40, 300])
@pytest.mark.parametrize("low", [-560.0, -700.0, -720.0, -745.0, -900.0, -30000.0, -3e38])
def test_shares_of_probabilities_below_the_least_number(moe, tokens, experts, low):
    rng = np.random.default_rng(2)
    scores = (low + rng.uniform(-3, 0, experts)).astype(np.float32)
    weights, ids = run(moe, tokens, scores, 8, scoring="sigmoid", scale=2.5)
    at = order(scores.astype(np.float64))[:8]
    assert ids.tolist() == at.tolist()
    assert np.abs(weights / (2.5 * shares(scores, at)) - 1).max() <= TOL
    # Softmax: one expert has it all, and a bias brings others forward.
    scores[11] = 0.0
    bias = torch.zeros(experts)
    bias[11] = -2.0
    bias[20:26] = 1.0
    weights, ids = run(moe, tokens, scores, 6, bias)
    at = np.arange(20, 26)
    assert sorted(ids.tolist()) == at.tolist()
    assert np.abs(weights / shares(scores, ids) - 1).max() <= TOL
    # With it among them there is a sum, and the others' shares are zero in f32.
    weights, ids = run(moe, tokens, scores, 7, bias * 0)
    assert ids[0] == 11 and weights.tolist() == [1.0] + [0.0] * 6


def test_shares_of_scores_at_minus_infinity(moe):
    scores = np.full(20, -INF, dtype=np.float32)
    weights, ids = run(moe, 3, scores, 4, scoring="sigmoid")
    assert ids.tolist() == [0, 1, 2, 3] and weights.tolist() == [0.25] * 4
    scores[[5, 9]] = -800.0
    weights, ids = run(moe, 3, scores, 4, scoring="sigmoid")
    assert ids.tolist() == [5, 9, 0, 1] and weights.tolist() == [0.5, 0.5, 0.0, 0.0]
    weights, ids = run(moe, 3, scores, 4, scoring="sigmoid", renormalize=False)
    assert weights.tolist() == [0.0] * 4
