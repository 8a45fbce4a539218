"""Pins of the oracle's distillation where the teacher's list is complete."""
import numpy as np
import pytest

import oracle as O


@pytest.mark.parametrize("masked", [-np.inf, -3.4028234663852886e38])
@pytest.mark.parametrize("allowed", [1, 2, 3, 10, 20, 128])
def test_complete_lists_give_the_divergence_of_the_listed_tokens(allowed, masked):
    """Log probabilities rounded to fp32 leave a mass of 1 - d, |d| within the rounding of the list (2^-19 + 2^-22 H).
    With p = (1 - d) p', log p = log p' + log(1 - d): sum p (log p - log q) differs from the divergence D of p' by
    (1 - d) log(1 - d) - d D, below 2 |d| (1 + D)."""
    r = np.random.default_rng([102, allowed])
    V, n = 300, 200
    x = np.full((2, n, V), masked)
    for i in range(n):
        at = r.permutation(V)[:allowed]
        x[:, i, at] = 2.5 * r.standard_normal((2, allowed))
    top = O.token_logprobs(x[0], None, allowed)
    lps = top["top_logprob"].astype(np.float32)
    o = O.distill_topk(x[1], top["top_id"], lps)
    lq = O.token_logprobs(x[1], None, 0)["lse"]
    for i in range(n):
        lp = top["top_logprob"][i]
        p = np.exp(lp)
        z = x[1, i, top["top_id"][i]]
        q = z - z.max() - np.log(np.exp(z - z.max()).sum())
        want, d = (p * (lp - q)).sum(), 2.0 ** -19 + 2.0 ** -22 * np.abs(p * lp).sum()
        assert abs(o["loss"][i] - want) <= 2 * d * (1 + abs(want)), (i, o["loss"][i], want)
        assert np.isfinite(o["grad"][i]).all() and np.all(o["grad"][i][x[1, i] == masked] == 0)
    assert np.isfinite(lq).all()


def test_the_loss_is_continuous_where_the_residue_stops_counting():
    """A residue within the rounding counts while the student's tail is at least as large: as the tail falls through
    it the loss does not jump.  On both sides of the point the loss differs from the listed part by p_r log(p_r / q_r)
    or nothing, |p_r log(p_r / q_r)| <= 1.1 p_r |1 - q_r / p_r| for a ratio within 10 % of one."""
    lps = np.log(np.array([[0.6, 0.4 - 1.0e-6]])).astype(np.float32)
    ids = np.array([[0, 1]])
    pr = 1 - np.exp(lps.astype(np.float64)).sum()
    assert 0 < pr < 2.0 ** -19
    losses = []
    for f in (0.95, 0.99, 1.01, 1.05):
        q = f * pr
        x = np.log(np.array([[0.6 * (1 - q), 0.4 * (1 - q), q]]))
        losses.append(O.distill_topk(x, ids, lps)["loss"][0])
    listed = (np.exp(lps.astype(np.float64)) * (lps - np.log([[0.6, 0.4]]))).sum()
    assert np.all(np.abs(np.array(losses) - listed) <= 1.1 * 0.05 * pr + 1.2 * pr)
    assert abs(losses[1] - losses[2]) <= 0.1 * pr


def test_a_residue_above_the_rounding_counts():
    x = np.array([[1.0, 0.5, -np.inf], [1.0, 0.5, -np.inf]])
    lps = np.log(np.array([[0.6, 0.3999], [0.6, 0.4]])).astype(np.float32)
    o = O.distill_topk(x, np.array([[0, 1], [0, 1]]), lps)
    assert o["loss"][0] == np.inf and np.isfinite(o["loss"][1])
