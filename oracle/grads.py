"""Training-side operators: float64 CPU oracle.

TEST INFRASTRUCTURE ONLY -- imported by ``tests/``, never by the product path.
It shares no code with the HIP library.  Plain definitions, row by row:

* ``policy_loss``: clipped policy loss with a KL term and its gradient with
  respect to the logits.
* ``lora_grad``: gradients of base + s (X A^T) B^T with one adapter per row.
"""
from __future__ import annotations

import numpy as np

__all__ = ["policy_loss", "lora_grad"]


def policy_loss(logits, targets, old, advantage, ref=None, clip_low=0.2, clip_high=0.2, kl_coef=0.0, temperature=1.0,
                weight=None) -> dict:
    """loss, logprob, ratio, kl (n,) and grad (n, V) of sum(weight * loss); logits (n, V) float64."""
    n, V = logits.shape
    out = {k: np.zeros(n) for k in ("loss", "logprob", "ratio", "kl")}
    out["grad"] = np.zeros((n, V))
    for i in range(n):
        w = 1.0 if weight is None else float(weight[i])
        t = int(targets[i])
        if not 0 <= t < V:
            continue
        x = np.asarray(logits[i], dtype=np.float64)
        if np.isnan(x).any() or np.isposinf(x).any() or np.isneginf(x).all():
            for k in ("loss", "logprob", "ratio", "kl"):
                out[k][i] = np.nan
            out["grad"][i] = 0.0 if w == 0.0 else np.nan
            continue
        z = x / temperature
        m = z.max()
        e = np.exp(z - m)
        others = e[:t].sum() + e[t + 1:].sum()
        total = others + e[t]
        lp = -np.log1p(others) if z[t] == m else (z[t] - m) - np.log(total)   # a sure token's is not rounded away
        a = float(advantage[i])
        with np.errstate(over="ignore", invalid="ignore", divide="ignore"):
            gone, o = lp == -np.inf, float(old[i])            # a masked token: ratio 0, whatever the behaviour's was
            r = 0.0 if gone and o == o else np.exp(lp - o)
            free, held = r * a, min(max(r, 1.0 - clip_low), 1.0 + clip_high) * a
            loss, c = (-held, 0.0) if free > held else (-free, -free)
            kl = 0.0
            if ref is not None:
                d = np.inf if gone and ref[i] == ref[i] else float(ref[i]) - lp
                kl = np.inf if d == np.inf else np.expm1(d) - d
                if kl_coef > 0:
                    loss = loss + kl_coef * kl
                    c = c - kl_coef * np.expm1(d)
        out["loss"][i], out["logprob"][i], out["ratio"][i], out["kl"][i] = loss, lp, r, kl
        if gone and c == c:                    # nor has it a gradient; a NaN stays
            c = 0.0
        g = -e / total
        g[t] = others / total
        out["grad"][i] = 0.0 if w == 0.0 else w * c * g / temperature
    return out


def lora_grad(X, dY, A, B, adapter, scale=None, base=None) -> dict:
    """dA, dB and dX; X (M, d_in), dY (M, d_out), A (n, r, d_in), B (n, d_out, r) float64; adapter outside [0, n): none."""
    n = A.shape[0]
    out = {"dA": np.zeros(A.shape), "dB": np.zeros(B.shape),
           "dX": np.zeros(X.shape) if base is None else np.array(base, dtype=np.float64)}
    for m in range(X.shape[0]):
        a = int(adapter[m])
        if 0 <= a < n:
            s = 1.0 if scale is None else float(scale[a])
            u, t = s * (dY[m] @ B[a]), s * (A[a] @ X[m])
            out["dA"][a] += np.outer(u, X[m])
            out["dB"][a] += np.outer(dY[m], t)
            out["dX"][m] += u @ A[a]
    return out
