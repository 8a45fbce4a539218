"""Seeded rows of logits, teacher lists and adapters, and the forward error
bounds (derived from the formulas, fp32 unit roundoff u = 2^-24) that the GPU
results are held to."""
import numpy as np

U = 2.0 ** -24
LOWEST = {"f32": -3.4028234663852886e38, "f16": -65504.0, "bf16": -3.3895313892515355e38}


def store(x, dtype):
    """float64/float32 values -> storage array of the type (bf16 as uint16 bits)."""
    x = np.asarray(x, dtype=np.float32)
    if dtype == "f32":
        return x.copy()
    if dtype == "f16":
        with np.errstate(over="ignore"):
            return x.astype(np.float16)
    u = x.view(np.uint32).astype(np.uint64)
    r = ((u + 0x7FFF + ((u >> 16) & 1)) >> 16).astype(np.uint16)
    return np.where(np.isnan(x), np.uint16(0x7FC0), r)


def exact(s, dtype):
    """Storage array -> the float64 values it stands for."""
    if dtype != "bf16":
        return s.astype(np.float64)
    return (s.astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def to_torch(s, dtype):
    import torch
    if dtype == "bf16":
        return torch.from_numpy(s.view(np.int16)).cuda().view(torch.bfloat16)
    return torch.from_numpy(s).cuda()


ROW_KINDS = ["plain", "peaked", "equal", "dead", "lowest", "lowest_but_one", "few", "ascending", "descending",
             "run", "zeros", "far", "large", "masked", "spread"]


def row(kind, V, dtype, r):
    """One row of logits as float32 values (rounded to the type by the caller)."""
    x = r.standard_normal(V).astype(np.float32) * 2.5
    if kind == "peaked":
        x[r.integers(0, V, 3)] += 20
    elif kind == "equal":
        x[:] = 1.5
    elif kind == "dead":
        x[:] = -np.inf
    elif kind == "lowest":
        x[:] = LOWEST[dtype]
    elif kind == "lowest_but_one":
        x[:] = LOWEST[dtype]
        x[V // 2] = 0.25
    elif kind == "few":
        keep = r.integers(0, V, 3)
        v = x[keep]
        x[:] = -np.inf
        x[keep] = v
    elif kind == "ascending":
        x = np.linspace(-10, 10, V).astype(np.float32)
    elif kind == "descending":
        x = np.linspace(10, -10, V).astype(np.float32)
    elif kind == "run":
        x[V // 3: V // 3 + 300] += 12
    elif kind == "zeros":
        x = np.where(np.arange(V) % 3 == 0, np.float32(-0.0), np.float32(0.0)).astype(np.float32)
    elif kind == "far":
        x[:] -= 3.0e4
        x[V // 4] = -2.0e4
    elif kind == "large":
        x *= 1.0e4 if dtype == "f16" else 2.0e37
    elif kind == "masked":
        x[r.random(V) < 0.9] = -np.inf
    elif kind == "spread":
        x *= 12
    return x


def rows(kinds, V, dtype, seed):
    r = np.random.default_rng([91, seed, V])
    return store(np.stack([row(k, V, dtype, r) for k in kinds]), dtype)


def steps(V):
    """Additions in a row on the way to a sum of V terms, at most: each lane adds
    a run of at most V / 64 + 8 terms, then pairs are joined."""
    return V / 64.0 + 8 + 40


def logprob_bounds(x, lse, T):
    """Bounds of lse, log probabilities and entropy per row: z - m carries three
    roundings of its size, e^(z - m) two units and its exponent's error, the sum
    one rounding per addition; the entropy's second sum the same on terms of
    size p |z - m|."""
    n = steps(x.shape[1])
    with np.errstate(invalid="ignore"):
        m = np.where(np.isfinite(x), x, -np.inf).max(1)
        z = np.where(np.isfinite(x), (x - m[:, None]) / T, -np.inf)
    p = np.exp(z)
    log_s = np.log(np.maximum(p.sum(1), 1.0))
    p = p / np.maximum(p.sum(1, keepdims=True), 1e-300)
    spread = np.where(p > 0, p * np.abs(np.where(np.isfinite(z), z, 0.0)), 0.0).sum(1)
    s_err = U * (n + 4 + 4 * spread)                      # relative error of S, absolute of log S
    base = s_err + 2 * U * (1 + log_s)
    lse = base + 3 * U * np.abs(np.where(np.isfinite(lse), m, 0.0) / T)
    ent = 2 * s_err * (1 + spread) + 4 * U * (1 + log_s)
    second = np.where(p > 0, p * np.where(np.isfinite(z), z, 0.0) ** 2, 0.0).sum(1)
    ent = ent + 6 * U * second                            # exponents' errors inside the weighted sum
    return base, lse, ent


def value_bound(base, lp):
    """Bound of a log probability next to the row's: the distance z - m again."""
    return base[:, None] + 5 * U * (1 + np.abs(np.nan_to_num(lp, neginf=0.0)) * 1.0) + 5 * U * np.abs(
        np.nan_to_num(lp, neginf=0.0))


def teacher(x, k, T, seed, pad=False):
    """Teacher lists of rows x (float64): the k best of a perturbed row."""
    r = np.random.default_rng([92, seed, x.shape[1], k])
    n, V = x.shape
    t = np.where(np.isfinite(x), x, 0.0) * 1.1 + r.standard_normal(x.shape)
    t = np.clip(t, -1e4, 1e4) / T
    ids = np.argsort(-t, axis=1, kind="stable")[:, :k]
    lse = t.max(1) + np.log(np.exp(t - t.max(1, keepdims=True)).sum(1))
    lp = np.take_along_axis(t, ids, 1) - lse[:, None]
    ids, lp = ids.astype(np.int32), lp.astype(np.float32)
    if pad:
        ids[0::3, k // 2:] = -1
        lp[1::3, k // 2:] = -np.inf
        if k > 2:
            ids[2::5, k - 1] = ids[2::5, 0]               # an id that comes twice
    return ids, lp


def distill_bounds(x, ids, lps, T, tail, weight, out, dtype):
    """Bounds of loss and gradient: p carries its exponent's error and two units,
    p_r = 1 - sum p the errors of the p and one rounding per term, the two sums
    of the student's row one rounding per addition and their exponents'.  What
    is below fp32's normal range may come out as zero."""
    n, V = x.shape
    c = steps(V) + 8
    loss_b, grad_b = np.zeros(n), np.zeros((n, V))
    ru = {"f32": U, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}[dtype]
    tiny = {"f32": 0.0, "f16": 2.0 ** -25, "bf16": 0.0}[dtype]
    for i in range(n):
        if not np.isfinite(x[i]).any() or np.isnan(x[i]).any() or np.isposinf(x[i]).any():
            continue
        live = {}
        for t, l in zip(ids[i], lps[i]):
            if 0 <= t < V and l != -np.inf and int(t) not in live:
                live[int(t)] = float(l)
        if not live:
            continue
        at, l = np.array(list(live)), np.array(list(live.values()))
        z = x[i] / T
        m = z.max()
        e = np.exp(z - m)
        lse = np.log(e.sum())                             # above m
        lq = (z - m) - lse
        q = np.exp(lq)
        zm = np.abs(np.where(np.isfinite(z), z - m, 0.0))
        s_err = U * (c + 4 * (q * zm).sum())
        if not tail:
            l = l - (l.max() + np.log(np.exp(l - l.max()).sum()))
        p = np.exp(l)
        p_err = p * U * (8 + len(p) + 4 * np.abs(l))
        lq_at = np.where(np.isfinite(lq[at]), lq[at], 0.0)
        b = (p * (s_err + U * (8 + 6 * np.abs(l) + 6 * np.abs(lq_at)))).sum()
        b += (p_err * (np.abs(l) + np.abs(lq_at) + 1)).sum() + U * len(p) * np.abs(p * (l - lq_at)).sum()
        g = q * (s_err + U * (8 + 4 * zm))
        inside = np.zeros(V, dtype=bool)
        inside[at] = True
        g[at] += p_err
        if tail:
            pr = max(0.0, 1.0 - p.sum())
            d_pr = p_err.sum() + U * (len(p) + 2)
            zr = np.where(inside, -np.inf, z)
            if np.isfinite(zr).any():
                mr = zr.max()
                er = np.exp(zr - mr)
                soft = er / er.sum()
                zrm = np.where(np.isfinite(zr), np.abs(zr - mr), 0.0)
                r_err = U * (c + 4 * (soft * zrm).sum())
                lqr = (mr - m) + np.log(er.sum()) - lse
                b += d_pr * (np.abs(np.log(max(pr, d_pr))) + np.abs(lqr) + 2)
                b += pr * (r_err + s_err + U * (8 + 6 * np.abs(lqr) + 4 * np.abs(mr - m)))
                g = g + soft * (d_pr + pr * (r_err + U * (10 + 4 * zrm)))
        w = 1.0 if weight is None else abs(float(weight[i]))
        loss_b[i] = b
        grad_b[i] = w / T * (g + 3 * U * np.abs(out["grad"][i]) * T / max(w, 1e-30))
        grad_b[i] += ru * (np.abs(out["grad"][i]) + grad_b[i]) + tiny + 4 * w / T * 2.0 ** -126
    return loss_b, grad_b


def adapters(M, d_in, d_out, rank, n, dtype, seed):
    r = np.random.default_rng([93, seed, M, d_in, d_out, rank, n])
    X = store(r.standard_normal((M, d_in)), dtype)
    A = store(r.standard_normal((n, rank, d_in)) / np.sqrt(d_in), dtype)
    B = store(r.standard_normal((n, d_out, rank)) * 0.3, dtype)
    s = r.uniform(0.5, 2.0, n).astype(np.float32)
    return X, A, B, s


def lora_bound(X, A, B, adapter, scale, Y, x_dtype, y_dtype):
    """Bound per output: the first product one rounding per addition, T rounded
    to two 16-bit terms (2^-16 of it in bf16, 2^-21 in fp16), the second product
    and the base one rounding per addition, one rounding to Y's type."""
    M, d_in = X.shape
    r = A.shape[1]
    out = np.zeros_like(Y)
    split = {"bf16": 2.0 ** -16, "f16": 2.0 ** -21}[x_dtype]
    tiny = {"bf16": 0.0, "f16": 2.0 ** -24}[x_dtype]      # the second fp16 term may be subnormal
    for m in range(M):
        a = int(adapter[m])
        if 0 <= a < A.shape[0]:
            s = 1.0 if scale is None else abs(float(scale[a]))
            tm = np.abs(A[a]) @ np.abs(X[m])
            t_err = s * tm * U * (d_in + 8) + s * np.abs(A[a] @ X[m]) * split + tiny
            out[m] = np.abs(B[a]) @ (t_err + s * np.abs(A[a] @ X[m]) * U * (2 * r + 8))
    ru = {"f32": 2 * U, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}[y_dtype]
    return out + ru * (np.abs(Y) + out) + ({"f16": 2.0 ** -25}.get(y_dtype, 0.0))
