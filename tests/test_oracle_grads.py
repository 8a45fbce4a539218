"""Pins of the training-side oracle: hand-worked rows, gradients against differences of the losses."""
import numpy as np

from oracle import grads as F


def test_policy_row_by_hand():
    # two tokens, logits 0 and ln 3: q = 1/4, 3/4
    x = np.array([[0.0, np.log(3.0)]] * 4)
    old = np.log([0.75, 0.75, 0.5, 0.25])
    adv = np.array([2.0, -2.0, 1.0, 1.0])
    o = F.policy_loss(x, [1, 1, 1, 1], old, adv, clip_low=0.2, clip_high=0.3)
    np.testing.assert_allclose(o["logprob"], np.log(0.75), rtol=1e-15)
    np.testing.assert_allclose(o["ratio"], [1, 1, 1.5, 3], rtol=1e-12)
    np.testing.assert_allclose(o["loss"], [-2, 2, -1.3, -1.3], rtol=1e-12)   # the last two are held at 1.3
    np.testing.assert_allclose(o["grad"][0], [2 * 0.25, -2 * 0.25], rtol=1e-12)
    np.testing.assert_array_equal(o["grad"][2:], 0)
    # a negative advantage is held from below, and never from above
    o = F.policy_loss(x[:2], [1, 1], np.log([3.0, 0.25]), np.array([-1.0, -1.0]))
    np.testing.assert_allclose(o["loss"], [0.8, 3.0], rtol=1e-12)
    assert not o["grad"][0].any() and o["grad"][1].any()


def test_kl_term_is_zero_at_the_reference_and_positive_elsewhere():
    x = np.random.default_rng(1).standard_normal((5, 9))
    lp = F.policy_loss(x, [3] * 5, np.zeros(5), np.zeros(5))["logprob"]
    o = F.policy_loss(x, [3] * 5, lp, np.zeros(5), ref=lp, kl_coef=0.5)
    assert np.abs(o["loss"]).max() < 1e-15 and np.abs(o["grad"]).max() < 1e-15
    assert np.all(F.policy_loss(x, [3] * 5, lp, np.zeros(5), ref=lp + [-1, -.1, .1, 1, 2], kl_coef=0.5)["kl"] > 0)


def test_policy_gradient_by_differences():
    r = np.random.default_rng(2)
    x, t = r.standard_normal((6, 11)) * 2, [0, 3, 10, -100, 5, 11]
    lp = F.policy_loss(x, t, np.zeros(6), np.zeros(6), temperature=0.7)["logprob"]
    kw = dict(old=lp + r.uniform(-.4, .4, 6), advantage=r.standard_normal(6), ref=lp + r.uniform(-1, 1, 6), kl_coef=0.3,
              temperature=0.7, weight=r.uniform(.5, 2, 6))
    o = F.policy_loss(x, t, **kw)
    assert not o["grad"][[3, 5]].any() and not o["loss"][[3, 5]].any()
    h = 1e-6
    for j in range(11):
        d = np.zeros_like(x)
        d[:, j] = h
        num = (F.policy_loss(x + d, t, **kw)["loss"] - F.policy_loss(x - d, t, **kw)["loss"]) / (2 * h)
        np.testing.assert_allclose(o["grad"][:, j], num * kw["weight"], atol=1e-8, rtol=1e-6)


def test_adapter_gradients_by_differences():
    r = np.random.default_rng(3)
    X, dY = r.standard_normal((7, 5)), r.standard_normal((7, 4))
    A, B, ad, s = r.standard_normal((2, 3, 5)), r.standard_normal((2, 4, 3)), [0, 1, 1, -1, 0, 2, 1], np.array([0.5, 2.0])
    g = F.lora_grad(X, dY, A, B, ad, s)

    def f(X, A, B):
        return sum(float(s[a] * (B[a] @ (A[a] @ X[m])) @ dY[m]) for m, a in enumerate(ad) if 0 <= a < 2)
    for name, i, v in (("dX", 0, X), ("dA", 1, A), ("dB", 2, B)):
        for at in [tuple(r.integers(0, n) for n in v.shape) for _ in range(12)]:
            args = [X, A, B]
            num = 0.0
            for sign in (1, -1):
                args[i] = v.copy()
                args[i][at] += sign * 1e-4
                num += sign * f(*args) / 2e-4
            np.testing.assert_allclose(g[name][at], num, rtol=1e-6, atol=1e-9)
