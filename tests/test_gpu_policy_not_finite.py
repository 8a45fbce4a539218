"""What is not finite in the policy loss: NaN and infinities in the behaviour, the advantage and the reference.

Rows whose softmax is one half each for two tokens, or nothing for a masked target, so that every number has a plain value:
each output is rounded once and made by a few fp32 functions of two units at most (8 roundings, 2^-24 each, in all)."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
LOW, HIGH = 1.0 - float(np.float32(0.2)), 1.0 + float(np.float32(0.2))
INF, NAN = np.inf, np.nan


def call(x, t, old, adv, ref=None, beta=0.0, weight=None, dtype="float32"):
    import torch
    from post_weight_quantization_08_amd import pipeline as P

    def dev(v):
        return torch.from_numpy(np.ascontiguousarray(v, dtype=np.float32)).cuda() if v is not None else None
    out = P.policy_loss(dev(x).to(getattr(torch, dtype)), torch.from_numpy(np.asarray(t, dtype=np.int32)).cuda(), dev(old),
                        dev(adv), ref_logprob=dev(ref), kl_coef=beta, weight=dev(weight))
    return {k: v.double().cpu().numpy() for k, v in out.items()}


def definition(lp, old, adv, ref, beta):
    """loss, ratio, kl and dloss/dl of one row in float64."""
    with np.errstate(all="ignore"):
        gone = lp == -INF
        ratio = 0.0 if gone and old == old else np.exp(lp - old)
        held = (LOW if ratio < LOW else HIGH if ratio > HIGH else ratio) * adv
        free = 0.0 if adv == 0 and ratio == INF else ratio * adv
        loss, c = (-held, 0.0) if free > held else (-free, -free)
        kl = 0.0
        if ref is not None:
            d = INF if gone and ref == ref else ref - lp
            up = np.expm1(d)
            kl = INF if d == INF else up - d if abs(d) > 0.1 else sum(d ** k / np.prod(np.arange(1.0, k + 1)) for k in range(12, 1, -1))
            if beta > 0:
                loss, c = loss + beta * kl, c - beta * up
        if gone and c == c:
            c = 0.0
    return loss, ratio, kl, c


def same(got, want, rel, what):
    """Equal where not finite (NaN with NaN), else within `rel`."""
    with np.errstate(over="ignore"):
        want = np.where(np.abs(want) > 3.4028235e38, np.sign(want) * INF, want)
    np.testing.assert_array_equal(np.isnan(got), np.isnan(want), err_msg=what)
    fine = np.isfinite(want)
    rest = ~fine & ~np.isnan(want)
    np.testing.assert_array_equal(got[rest], want[rest], err_msg=what)
    bad = np.abs(got[fine] - want[fine]) > rel * np.abs(want[fine]) + 2.0 ** -149
    assert not bad.any(), (what, got[fine][bad][:4], want[fine][bad][:4])


SPECIAL = [(o, a, r) for o in (NAN, INF, -INF, -1.0) for a in (1.0, -1.0, 0.0, NAN, INF) for r in (NAN, INF, -INF, -1.2)]


@pytest.mark.parametrize("V", [2, 40000])
@pytest.mark.parametrize("beta", [0.0, 0.1])
@pytest.mark.parametrize("masked", [False, True])
def test_what_is_not_finite(V, beta, masked):
    """NaN and infinities in the behaviour, the advantage and the reference, against a scored and a masked target: by the
    formula, a NaN never turned into a number, nothing in a row of weight 0."""
    n = 2 * len(SPECIAL)
    old, adv, ref = (np.tile(np.array(v), 2) for v in zip(*SPECIAL))
    weight = np.repeat([1.0, 0.0], len(SPECIAL))
    x = np.full((n, V), -INF)
    x[:, 0] = 0.0
    x[:, V - 1] = -INF if masked else 0.0
    g = call(x, np.full(n, V - 1), old, adv, ref, beta, weight)
    lp = -INF if masked else -np.log(2.0)
    want = np.array([definition(lp, o, a, r, float(np.float32(beta))) for o, a, r in zip(old, adv, ref)])
    for i, name in enumerate(("loss", "ratio", "kl")):
        same(g[name], want[:, i], 8 * U, name)
    c, grad = want[:, 3], g["grad"]
    live = weight > 0
    assert not grad[~live].any()
    np.testing.assert_array_equal(np.isnan(grad[live]).all(1), np.isnan(c[live]))
    finite = live & np.isfinite(c)
    share = 0.0 if masked else 0.5
    same(grad[finite][:, V - 1], c[finite] * share, 8 * U, "gradient of the target")
    same(grad[finite][:, 0], -c[finite] * share, 8 * U, "gradient of the other token")
    assert not grad[finite][:, 1:V - 1].any()
