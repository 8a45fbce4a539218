"""A scored row's own numbers in the policy loss are 64-bit numbers.

Rows of two tokens at logit 0 have the log probability -ln 2 and a sum that fp32 holds exactly, so what is left of the error
is the row's numbers: 64-bit differences and functions of them (below 2^-40 here), each output rounded once to fp32 (half a
step, 2^-24) and the gradient's element in a few fp32 products (8 roundings at most)."""
import numpy as np
import pytest

from tests.test_gpu_policy_not_finite import U, call, definition, same

pytestmark = pytest.mark.gpu


def test_numbers_keep_their_digits():
    """Ratios, KL terms, losses and gradients within half a step, for differences from 1e-6 to 88."""
    r = np.random.default_rng(3)
    n = 4000
    lp = -np.log(2.0)
    size = 10.0 ** r.uniform(-6, np.log10(88.0), n) * r.choice([-1, 1], n)
    old, ref = np.full(n, lp), np.full(n, lp)
    old[:n // 2] = lp - size[:n // 2]
    ref[n // 2:] = lp + size[n // 2:]
    old, ref = old.astype(np.float32).astype(np.float64), ref.astype(np.float32).astype(np.float64)
    adv = -r.uniform(0.5, 2, n).astype(np.float32).astype(np.float64)       # the free side above the interval
    g = call(np.zeros((n, 2)), np.ones(n), old, adv, ref, 0.25)
    want = np.array([definition(lp, o, a, f, 0.25) for o, a, f in zip(old, adv, ref)])
    same(g["logprob"], np.full(n, lp), 1.01 * U, "logprob")
    for i, name in enumerate(("loss", "ratio")):
        same(g[name], want[:, i], 1.01 * U, name)
    # an error e of l moves kl by (e^d - 1) e, which is 2 e / d of it for small d; in half of the rows ref is l rounded
    # to fp32 and d no more than 2e-9.  e: l's 64 bits here and there, 2^-50 at most (l has units of 2^-53)
    up = np.abs(np.expm1(ref - lp))
    assert np.all(np.abs(g["kl"] - want[:, 2]) <= 1.01 * U * want[:, 2] + 2.0 ** -50 * up)
    # the coefficient may be a difference: its units are those of the parts
    parts = np.abs(adv * want[:, 1]) + 0.25 * up
    assert np.all(np.abs(g["grad"][:, 1] - 0.5 * want[:, 3]) <= 8 * U * (np.abs(want[:, 3]) + 1e-6 * parts))


def test_numbers_beyond_fp32_on_the_way():
    """A ratio or e^(ref - l) above fp32's largest number, times a small factor, is a number that fp32 holds."""
    lp = -np.log(2.0)
    old = np.array([-95.0, -100.0, -140.0, -1.0, -1.0, -1.0], dtype=np.float32).astype(np.float64)
    adv = np.array([-1e-12, -1e-20, -1e-30, 1.0, 1.0, -1.0], dtype=np.float32).astype(np.float64)
    ref = np.array([-1.0, -1.0, -1.0, 88.5, 92.0, 95.0], dtype=np.float32).astype(np.float64)
    beta = float(np.float32(1e-9))
    g = call(np.zeros((6, 2)), np.ones(6), old, adv, ref, beta)
    want = np.array([definition(lp, o, a, f, beta) for o, a, f in zip(old, adv, ref)])
    assert np.isfinite(want[:, 0]).all() and np.isinf(g["ratio"][:3]).any() and np.isinf(g["kl"][3:]).any()
    for i, name in enumerate(("loss", "ratio", "kl")):
        same(g[name], want[:, i], 1.01 * U, name)
    same(g["grad"][:, 1], 0.5 * want[:, 3], 8 * U, "gradient")


def test_log_probabilities_far_from_the_behaviour():
    """Differences of 1e30, to the fp32 numbers next to l and to l with fewer digits: the ratio is 0 or infinite, never below."""
    x = np.zeros((4, 2), dtype=np.float32)
    x[:, 1] = -2.88e37 * np.array([1, 1, 1.7, 1.7])
    lp = x[:, 1].astype(np.float64)
    old = np.array([np.nextafter(x[0, 1], np.float32(s), dtype=np.float32) for s in (0, -np.inf)] + [x[2, 1] * f for f in (0.9, 1.1)])
    g = call(x, np.ones(4), old, np.full(4, -1.5), old, 0.1)
    np.testing.assert_array_equal(g["logprob"], lp)
    np.testing.assert_array_equal(g["ratio"], [0, np.inf, 0, np.inf])
    want = [definition(p, float(o), -1.5, float(o), 0.1) for p, o in zip(lp, old)]
    same(g["kl"], np.array([w[2] for w in want]), 1.01 * U, "kl")


@pytest.mark.parametrize("gap", [0.25, 3.0, 9.0, 20.0, 60.0])
def test_log_probability_of_two_tokens(gap):
    """-log(1 + e^(-gap)) above and below: the sum is one power of e, off by two units of fp32 and its exponent's two
    roundings (2 gap 2^-24); the result is rounded once."""
    x = np.zeros((2, 2), dtype=np.float32)
    x[0, 1], x[1, 1] = gap, -gap
    g = call(x, [1, 1], [0.0, 0.0], [1.0, 1.0])
    sure, other = -np.log1p(np.exp(-gap)), -gap - np.log1p(np.exp(-gap))
    err = np.exp(-gap) * U * (4 + 2 * gap)
    assert abs(g["logprob"][0] - sure) <= err + 1.01 * U * abs(sure)
    assert abs(g["logprob"][1] - other) <= err + 1.01 * U * abs(other)
