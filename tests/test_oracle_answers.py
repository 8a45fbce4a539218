"""Pins of the oracle of the answer-side operators: hand examples, brute-force
loops, and gradients against finite differences."""
import math

import numpy as np
import pytest

import oracle as O


def test_hand_example_logprobs():
    """Logits log 1, log 2, log 5 at T = 1: probabilities 1/8, 2/8, 5/8."""
    x = np.log(np.array([[1.0, 2.0, 5.0]]))
    o = O.token_logprobs(x, [1], 2)
    assert math.isclose(o["logprob"][0], math.log(2 / 8), rel_tol=1e-14)
    assert math.isclose(o["lse"][0], math.log(8), rel_tol=1e-14)
    h = -sum(p * math.log(p) for p in (1 / 8, 2 / 8, 5 / 8))
    assert math.isclose(o["entropy"][0], h, rel_tol=1e-13)
    assert o["top_id"][0].tolist() == [2, 1]
    np.testing.assert_allclose(o["top_logprob"][0], [math.log(5 / 8), math.log(2 / 8)], rtol=1e-13)


def test_ties_masks_and_broken_rows():
    x = np.array([[1.0, 3.0, 3.0, -0.0, 0.0], [-np.inf] * 5, [0, np.nan, 1, np.inf, 2], [0, 0, np.inf, 0, 0]])
    o = O.token_logprobs(x, [-100, 2, 0, 2], 4)
    assert o["top_id"][0].tolist() == [1, 2, 0, 3]
    assert o["logprob"][0] == 0.0                      # target outside: not scored
    assert o["lse"][1] == -np.inf and o["entropy"][1] == 0.0 and o["logprob"][1] == -np.inf
    assert o["top_id"][1].tolist() == [0, 1, 2, 3] and np.all(o["top_logprob"][1] == -np.inf)
    assert o["top_id"][2].tolist() == [1, 3, 4, 2] and np.all(np.isnan(o["top_logprob"][2]))
    assert np.isnan(o["lse"][3]) and np.isnan(o["entropy"][3]) and o["top_id"][3].tolist() == [2, 0, 1, 3]


@pytest.mark.parametrize("T", [0.5, 1.0, 3.0])
def test_uniform_rows_have_log_v(T):
    o = O.token_logprobs(np.full((1, 37), -7.25), [5], 3, T)
    assert math.isclose(o["entropy"][0], math.log(37), rel_tol=1e-13)
    assert math.isclose(o["logprob"][0], -math.log(37), rel_tol=1e-13)
    assert o["top_id"][0].tolist() == [0, 1, 2]


def _case(seed, n=3, V=11, k=4):
    r = np.random.default_rng([95, seed])
    x = r.standard_normal((n, V)) * 2
    ids = np.stack([r.permutation(V)[:k] for _ in range(n)])
    lp = np.log(r.dirichlet(np.ones(k), n) * r.uniform(0.4, 0.95, (n, 1)))
    return x, ids, lp


@pytest.mark.parametrize("T", [0.7, 1.0, 2.0])
@pytest.mark.parametrize("tail", [False, True])
def test_gradient_is_the_difference_quotient(T, tail):
    """Central differences of the loss; the third derivative of a log-sum-exp
    along one coordinate is below 1 / T^3 per unit of probability, so the
    truncation is below h^2 / T^3 (two such terms) and the rounding below
    1e-14 / h."""
    x, ids, lp = _case(1)
    w = np.array([0.5, 1.0, 2.0])
    g = O.distill_topk(x, ids, lp, T, tail, w)["grad"]
    h = 1e-4
    for i in range(x.shape[0]):
        for j in range(x.shape[1]):
            up, dn = x.copy(), x.copy()
            up[i, j] += h
            dn[i, j] -= h
            d = (O.distill_topk(up, ids, lp, T, tail)["loss"][i] - O.distill_topk(dn, ids, lp, T, tail)["loss"][i])
            assert abs(w[i] * d / (2 * h) - g[i, j]) < 2 * (h * h / T ** 3 + 1e-14 / h)


def test_loss_is_the_divergence_of_the_bucketed_distributions():
    x, ids, lp = _case(2, n=1)
    q = np.exp(x[0]) / np.exp(x[0]).sum()
    p = np.exp(lp[0])
    both = [(p[i], q[ids[0][i]]) for i in range(len(p))]
    both.append((1 - p.sum(), 1 - q[ids[0]].sum()))
    want = sum(a * math.log(a / b) for a, b in both)
    assert math.isclose(O.distill_topk(x, ids, lp, 1.0, True)["loss"][0], want, rel_tol=1e-12)
    pn = p / p.sum()
    want = sum(a * math.log(a / q[t]) for a, t in zip(pn, ids[0]))
    assert math.isclose(O.distill_topk(x, ids, lp, 1.0, False)["loss"][0], want, rel_tol=1e-12)


def test_a_student_equal_to_its_teacher_has_loss_and_gradient_zero():
    x, ids, _ = _case(3)
    full = O.token_logprobs(x, None, 4)
    o = O.distill_topk(x, full["top_id"], full["top_logprob"], 1.0, True)
    assert np.all(np.abs(o["loss"]) < 1e-14) and np.all(np.abs(o["grad"]) < 1e-14)


def test_padding_repeats_and_empty_lists():
    x, ids, lp = _case(4, n=1)
    a = O.distill_topk(x, ids[:, :2], lp[:, :2], 1.0, True)
    for pad_id, pad_lp in ((-1, -0.3), (11, -0.3), (5, -np.inf), (ids[0, 0], -0.01)):
        b = O.distill_topk(x, np.hstack([ids[:, :2], [[pad_id]]]), np.hstack([lp[:, :2], [[pad_lp]]]), 1.0, True)
        np.testing.assert_array_equal(a["grad"], b["grad"])
        assert a["loss"][0] == b["loss"][0]
    o = O.distill_topk(x, np.full((1, 3), -1), np.zeros((1, 3)), 1.0, True)
    assert o["loss"][0] == 0 and np.all(o["grad"] == 0)


def test_lora_by_hand():
    """One input channel pair, rank 1: (1, 2) . (3, 4) = 11, times 0.5, times (2, -1)."""
    X = np.array([[1.0, 2.0], [1.0, 2.0], [5.0, 5.0]])
    A = np.array([[[3.0, 4.0]], [[1.0, 0.0]]])
    B = np.array([[[2.0], [-1.0]], [[10.0], [20.0]]])
    Y = O.lora(X, A, B, [0, 1, -1], np.array([0.5, 2.0]), np.ones((3, 2)))
    np.testing.assert_array_equal(Y, [[12.0, -4.5], [21.0, 41.0], [1.0, 1.0]])
    np.testing.assert_array_equal(O.lora(X, A, B, [2, 0, 0])[0], [0.0, 0.0])
