"""Answer-side operators: float64 CPU oracle.

TEST INFRASTRUCTURE ONLY -- imported by ``tests/``, never by the product path.
It shares no code with the HIP library.  Plain definitions, row by row:

* ``token_logprobs``: log probabilities of given tokens, log-sum-exp, entropy
  and the k best alternatives (ties to the lower id) of rows of logits.
* ``distill_topk``: the loss of a student's row against a teacher's top list
  and its gradient with respect to the student's logits.
* ``lora``: base + scale (X A^T) B^T with one adapter per row.
"""
from __future__ import annotations

import numpy as np

__all__ = ["token_logprobs", "distill_topk", "lora"]


def token_logprobs(logits: np.ndarray, targets, k: int, temperature: float = 1.0) -> dict:
    """logits (n, V) float64 (exact values of any format), targets (n,) ints or None."""
    n, V = logits.shape
    out = {"logprob": np.zeros(n), "lse": np.zeros(n), "entropy": np.zeros(n),
           "top_logprob": np.zeros((n, k)), "top_id": np.zeros((n, k), dtype=np.int64)}
    for i in range(n):
        x = np.asarray(logits[i], dtype=np.float64)
        # descending, NaN first, equal values by index (a stable sort of the
        # negated values keeps the index order)
        rank = np.argsort(np.where(np.isnan(x), -np.inf, -x), kind="stable")
        if np.isnan(x).any():
            nan = np.flatnonzero(np.isnan(x))
            rest = rank[~np.isnan(x[rank])]
            rank = np.concatenate([nan, rest])
        if np.isnan(x).any() or np.isposinf(x).any():
            lse = ent = np.nan
            lp = np.full(V, np.nan)
        elif np.isneginf(x).all():
            lse, ent, lp = -np.inf, 0.0, np.full(V, -np.inf)
        else:
            z = x / temperature
            m = z.max()
            log_s = np.log(np.exp(z - m).sum())
            lse = m + log_s
            lp = (z - m) - log_s                  # the type's lowest value as m leaves log_s whole
            live = np.isfinite(lp)
            ent = -(np.exp(lp[live]) * lp[live]).sum()
        out["lse"][i], out["entropy"][i] = lse, ent
        out["top_id"][i] = rank[:k]
        out["top_logprob"][i] = lp[rank[:k]]
        if targets is not None and 0 <= targets[i] < V:
            out["logprob"][i] = lp[targets[i]]
    return out


def distill_topk(logits: np.ndarray, top_id: np.ndarray, top_logprob: np.ndarray, temperature: float = 1.0,
                 tail: bool = True, weight=None) -> dict:
    """loss (n,) and grad (n, V) of sum(weight * loss); logits (n, V) float64."""
    n, V = logits.shape
    loss, grad = np.zeros(n), np.zeros((n, V))
    for i in range(n):
        w = 1.0 if weight is None else float(weight[i])
        ids, lps = [], []
        for t, l in zip(top_id[i], top_logprob[i]):
            if 0 <= t < V and l != -np.inf and int(t) not in ids:
                ids.append(int(t))
                lps.append(float(l))
        if not ids:
            continue
        x = np.asarray(logits[i], dtype=np.float64)
        if np.isnan(x).any() or np.isposinf(x).any() or np.isneginf(x).all():
            loss[i] = np.nan
            grad[i] = 0.0 if w == 0.0 else np.nan
            continue
        ids, lps = np.array(ids), np.array(lps)
        z = x / temperature
        m = z.max()
        log_s = np.log(np.exp(z - m).sum())
        lq = (z - m) - log_s
        if not tail:
            lps = lps - (lps.max() + np.log(np.exp(lps - lps.max()).sum()))
        p = np.exp(lps)
        inside = np.zeros(V, dtype=bool)
        inside[ids] = True
        with np.errstate(divide="ignore", invalid="ignore"):
            terms = np.where(p > 0, p * (lps - lq[ids]), 0.0)
            total = terms.sum()
            g = np.exp(lq)
            if tail:
                pr = max(0.0, 1.0 - p.sum())
                zr = z[~inside]
                mr = zr.max() if zr.size else -np.inf
                sr = np.exp(zr - mr).sum() if mr > -np.inf else 0.0
                lqr = (mr - m) + np.log(sr) - log_s if sr > 0 else -np.inf
                # the rounding of a complete list's log probabilities is no mass that the student lacks
                if pr <= 2.0 ** -19 + 2.0 ** -22 * np.where(p > 0, p * np.abs(lps), 0.0).sum() and np.exp(lqr) < pr:
                    pr = 0.0
                if pr > 0:
                    total += pr * (np.log(pr) - lqr)
                # q_j (1 - p_r / q_r) = q_j - p_r softmax over the tail
                if mr > -np.inf:
                    g[~inside] -= pr * np.exp(zr - mr) / sr
        g[ids] -= p
        loss[i] = total
        grad[i] = 0.0 if w == 0.0 else w * g / temperature
    return {"loss": loss, "grad": grad}


def lora(X: np.ndarray, A: np.ndarray, B: np.ndarray, adapter, scale=None, base=None) -> np.ndarray:
    """X (M, d_in), A (n, r, d_in), B (n, d_out, r) float64; adapter (M,) ints, outside [0, n): none."""
    M = X.shape[0]
    Y = np.zeros((M, B.shape[1])) if base is None else np.array(base, dtype=np.float64)
    for m in range(M):
        a = int(adapter[m])
        if 0 <= a < A.shape[0]:
            Y[m] += (1.0 if scale is None else float(scale[a])) * (B[a] @ (A[a] @ X[m]))
    return Y
