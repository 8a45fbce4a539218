"""Workloads of training and serving in 8 bits beside the 4-bit layer: quantizing to
e4m3 with a power-of-two scale for each block of 128, the product of such operands,
the adapters' backward pass from 16-bit or 8-bit activations, and a clipped policy
loss with a KL term.

Each case names its operator in "op" and its sizes.  prepare() makes what a
program holds before the call; run() is one call, in plain torch operations
(32 bits, rounded once at the end) or, with `own` set, through the package;
exact() is the operator's definition in 64 bits.
"""
import math

import torch

own = False

_TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
_BLOCK = 128


def listed():
    return [
        # a layer's inputs of a training batch, kept in 8 bits for the backward pass
        {"name": "quantize_rows", "op": "quantize", "rows": 8192, "cols": 11008, "dtype": "bf16", "tiles": False},
        # the 70B-shaped up projection in 8 bits, with its transpose for the backward product
        {"name": "quantize_weights", "op": "quantize", "rows": 28672, "cols": 8192, "dtype": "bf16", "tiles": True},
        # one token of one request through an attention projection
        {"name": "matmul_one", "op": "matmul", "m": 1, "d_in": 4096, "d_out": 4096, "x": "f16", "y": "f16"},
        # a decode batch on the 70B-shaped up projection
        {"name": "matmul_batch", "op": "matmul", "m": 48, "d_in": 8192, "d_out": 28672, "x": "bf16", "y": "bf16"},
        # a prompt through a layer whose sizes fit nothing, fp32 on both sides
        {"name": "matmul_odd", "op": "matmul", "m": 777, "d_in": 11000, "d_out": 4001, "x": "f32", "y": "f32"},
        # a training batch whose inputs were quantized once
        {"name": "matmul_train", "op": "matmul", "m": 8192, "d_in": 8192, "d_out": 28672, "x": "e4m3", "y": "bf16"},
        # a short correction set, 16-bit activations, factors alone
        {"name": "grad_few", "op": "grad", "m": 96, "d_in": 4096, "d_out": 4096, "rank": 8, "adapters": 1, "x": "bf16",
         "factor": "bf16", "dy": "bf16", "dx": False},
        # eight adapters in one batch, half-precision training
        {"name": "grad_many", "op": "grad", "m": 2048, "d_in": 4096, "d_out": 14336, "rank": 16, "adapters": 8, "x": "f16",
         "factor": "f16", "dy": "f16", "dx": True},
        # a training batch of one adapter from 8-bit checkpoints, gradient passed on to the layer below
        {"name": "grad_train", "op": "grad", "m": 8192, "d_in": 11008, "d_out": 4096, "rank": 64, "adapters": 1, "x": "e4m3",
         "factor": "bf16", "dy": "bf16", "dx": True},
        # a few tokens of a short answer
        {"name": "policy_few", "op": "policy", "n": 8, "vocab": 32000, "dtype": "f32", "temp": 1.0, "kl": 0.05,
         "grad": True},
        # fp16 rows of odd length, answers sampled at 0.7
        {"name": "policy_odd", "op": "policy", "n": 777, "vocab": 50021, "dtype": "f16", "temp": 0.7, "kl": 0.0,
         "grad": True},
        # a training batch of answers of a large-vocabulary model
        {"name": "policy_train", "op": "policy", "n": 4096, "vocab": 131072, "dtype": "bf16", "temp": 1.0, "kl": 0.02,
         "grad": True},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["quantize", "matmul", "matmul", "grad", "grad", "policy"])
    if op == "quantize":
        return {"op": op, "rows": _log_int(rng, 1, 8192), "cols": _log_int(rng, 100, 14336),
                "dtype": rng.choice(["f32", "f16", "bf16"]), "tiles": rng.random() < 0.4}
    if op == "matmul":
        x = rng.choice(["e4m3", "bf16", "f16", "f32"])
        d_in = _log_int(rng, 200, 11008)
        return {"op": op, "m": _log_int(rng, 1, 8192), "d_in": -(-d_in // _BLOCK) * _BLOCK if x == "e4m3" else d_in,
                "d_out": _log_int(rng, 200, 14336), "x": x, "y": rng.choice(["f32", "f16", "bf16"])}
    if op == "grad":
        factor = rng.choice(["f16", "bf16"])
        x = rng.choice(["e4m3", factor])
        d_in = _log_int(rng, 200, 11008)
        return {"op": op, "m": _log_int(rng, 1, 8192), "d_in": d_in, "d_out": _log_int(rng, 200, 4096),
                "rank": rng.choice([4, 8, 16, 24, 32, 64]), "adapters": rng.choice([1, 1, 2, 5, 8]), "x": x,
                "factor": factor, "dy": rng.choice([factor, "f32"]), "dx": rng.random() < 0.6}
    dtype = rng.choice(["f32", "f16", "bf16"])
    return {"op": op, "n": _log_int(rng, 1, 2048 if dtype == "f32" else 4096), "vocab": _log_int(rng, 1000, 131072),
            "dtype": dtype, "temp": rng.choice([1.0, 0.7, 2.0]), "kl": rng.choice([0.0, 0.02, 0.1]),
            "grad": rng.random() < 0.8}


# ---------------------------------------------------------------- inputs
def _activations(rows, cols, gen):
    """Rows of different sizes with a few large channels."""
    x = torch.randn(rows, cols, generator=gen, device="cuda")
    x *= 0.2 + 2.0 * torch.rand(rows, 1, generator=gen, device="cuda")
    large = torch.randint(0, cols, (max(1, cols // 200),), generator=gen, device="cuda")
    x[:, large] *= 30.0
    return x


def _padded(n):
    return -(-n // _BLOCK) * _BLOCK


def _quantize(x, tiles=False):
    """(codes, scales as bytes) of rows in blocks of 128, or of 128 x 128 tiles: codes padded to whole blocks with
    zeros, the scale the smallest power of two at which the block's largest magnitude is at most 448."""
    rows, cols = x.shape
    x = torch.nn.functional.pad(x.float(), (0, _padded(cols) - cols))
    blocks = x.reshape(rows, -1, _BLOCK)
    top = blocks.abs().amax(2)
    if tiles:
        full = torch.nn.functional.pad(top, (0, 0, 0, _padded(rows) - rows))
        top = full.reshape(-1, _BLOCK, top.shape[1]).amax(1)
    b = (((top.view(torch.int32) + 0x1FFFFF) >> 23) - 8).clamp(min=27)
    back = ((254 - b) << 23).view(torch.float32)
    if tiles:
        back = back.repeat_interleave(_BLOCK, dim=0)[:rows]
    codes = (blocks * back[:, :, None]).reshape(rows, -1).to(torch.float8_e4m3fn)
    return codes, b.to(torch.uint8)


def _values(codes, b, tiles=False):
    s = (b.to(torch.int32) << 23).view(torch.float32)
    if tiles:
        s = s.repeat_interleave(_BLOCK, dim=0)[:codes.shape[0]]
    return (codes.float().reshape(codes.shape[0], -1, _BLOCK) * s[:, :, None]).reshape(codes.shape[0], -1)


def _prepare_matmul(case, gen):
    m, d_in, d_out = case["m"], case["d_in"], case["d_out"]
    w = torch.randn(d_out, d_in, generator=gen, device="cuda") / math.sqrt(d_in)
    w *= 0.3 + torch.rand(d_out, 1, generator=gen, device="cuda")
    s = {}
    s["W"], s["w_scales"] = _quantize(w, tiles=True)
    del w
    x = _activations(m, d_in, gen)
    if case["x"] == "e4m3":
        s["X"], s["x_scales"] = _quantize(x)
    else:
        s["X"], s["x_scales"] = x.to(_TYPES[case["x"]]), None
    return s


def _prepare_grad(case, gen):
    m, d_in, d_out, r, na = case["m"], case["d_in"], case["d_out"], case["rank"], case["adapters"]
    dt = _TYPES[case["factor"]]
    s = {"A": (torch.randn(na, r, d_in, generator=gen, device="cuda") / math.sqrt(d_in)).to(dt),
         "B": (torch.randn(na, d_out, r, generator=gen, device="cuda") * 0.3).to(dt),
         "scale": 0.5 + 1.5 * torch.rand(na, generator=gen, device="cuda")}
    x = _activations(m, d_in, gen)
    if case["x"] == "e4m3":
        s["X"], s["x_scales"] = _quantize(x)
    else:
        s["X"], s["x_scales"] = x.to(dt), None
    # what comes back: rows of different sizes, padding of nothing
    dy = torch.randn(m, d_out, generator=gen, device="cuda") * torch.rand(m, 1, generator=gen, device="cuda")
    if m > 1:
        dy *= (torch.rand(m, 1, generator=gen, device="cuda") >= 0.1)
    s["dY"] = dy.to(_TYPES[case["dy"]])
    if na > 1:
        # every request's tokens in a run, ragged lengths, one run without an adapter
        cut = torch.sort(torch.randint(0, m, (2 * na,), generator=gen, device="cuda")).values
        a = torch.searchsorted(cut, torch.arange(m, device="cuda"), right=True)
        s["adapter"] = torch.where(a == 1, torch.full_like(a, -1), a % na).to(torch.int32)
    else:
        s["adapter"] = torch.zeros(m, dtype=torch.int32, device="cuda")
    # the gradient that reached the layer's input through the frozen weights
    s["base"] = torch.randn(m, d_in, generator=gen, device="cuda").to(dt) if case["dx"] else None
    return s


def _prepare_policy(case, gen):
    n, v = case["n"], case["vocab"]
    x = torch.randn(n, v, generator=gen, device="cuda")
    x *= 1.0 + 2.0 * torch.rand(n, 1, generator=gen, device="cuda")
    at = torch.randint(0, v, (n, 1), generator=gen, device="cuda")
    at = (at + torch.arange(16, device="cuda") * (v // 16)) % v
    x.scatter_(1, at, 4.0 + 12.0 * torch.rand(n, 16, generator=gen, device="cuda"))
    # constrained positions: every eighth row keeps half of the vocabulary
    gone = torch.rand(n // 8 + 1, v, generator=gen, device="cuda") < 0.5
    x[::8].masked_fill_(gone[:x[::8].shape[0]], -math.inf)
    del gone
    logits = x.to(_TYPES[case["dtype"]])
    # the answer's tokens: sampled, as the behaviour that made them did
    x /= case["temp"]
    noise = torch.rand(n, v, generator=gen, device="cuda").clamp_(min=1e-20).log_().neg_().log_().neg_()
    targets = noise.add_(x).argmax(1)
    del noise
    lp = x.gather(1, targets[:, None])[:, 0] - torch.logsumexp(x, 1)
    del x
    # the behaviour's and the reference's log probabilities of the same tokens
    old = lp + 0.2 * torch.randn(n, generator=gen, device="cuda")
    ref = lp + 0.3 * torch.randn(n, generator=gen, device="cuda")
    if n > 1:
        targets = torch.where(torch.rand(n, generator=gen, device="cuda") < 0.1, torch.full_like(targets, -100), targets)
    # mean over the batch; fp16 gradients are kept in range by a loss scale
    return {"logits": logits, "targets": targets.to(torch.int32), "old": old, "ref": ref if case["kl"] > 0 else None,
            "advantage": torch.randn(n, generator=gen, device="cuda"),
            "weight": torch.full((n,), (4096.0 if case["dtype"] == "f16" else 1.0) / n, device="cuda")}


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    if case["op"] == "quantize":
        x = _activations(case["rows"], case["cols"], gen)
        if case["tiles"]:
            x /= math.sqrt(case["cols"])
        s = {"X": x.to(_TYPES[case["dtype"]])}
    elif case["op"] == "matmul":
        s = _prepare_matmul(case, gen)
    elif case["op"] == "grad":
        s = _prepare_grad(case, gen)
    else:
        s = _prepare_policy(case, gen)
    s["case"] = case
    s["keep"] = {}   # output buffers and workspace that a program reuses from call to call
    return s


# ---------------------------------------------------------------- the plain forms
def _scale_type(b):
    return b.view(torch.float8_e8m0fnu)


def _plain_quantize(s):
    tiles = s["case"]["tiles"]
    codes, b = _quantize(s["X"], tiles)
    out = {"codes": codes, "scales": _scale_type(b)}
    if tiles:
        # a tile's scale is the same both ways, so its transpose has the same codes
        t = torch.nn.functional.pad(codes.view(torch.uint8), (0, 0, 0, _padded(codes.shape[0]) - codes.shape[0]))
        out["codes_t"] = t.t()[:s["case"]["cols"]].contiguous().view(torch.float8_e4m3fn)
        out["scales_t"] = _scale_type(b.t().contiguous())
    return out


def _plain_matmul(s):
    c = s["case"]
    codes, b = (s["X"], s["x_scales"]) if c["x"] == "e4m3" else _quantize(s["X"])
    y = _values(codes, b) @ _values(s["W"], s["w_scales"], tiles=True).t()
    return y.to(_TYPES[c["y"]])


def _plain_grad(s):
    """The adapters side by side: one product with all of A, the other adapters' columns dropped."""
    c = s["case"]
    na, r, d_in = s["A"].shape
    d_out = s["B"].shape[1]
    x = _values(s["X"], s["x_scales"])[:, :d_in] if c["x"] == "e4m3" else s["X"].float()
    dy = s["dY"].float()
    mine = s["adapter"].long()[:, None] == torch.arange(na, device=x.device).repeat_interleave(r)[None, :]
    by = torch.where(mine, s["scale"].repeat_interleave(r)[None, :], torch.zeros((), device=x.device))
    a = s["A"].float().reshape(na * r, d_in)
    b = s["B"].float().permute(1, 0, 2).reshape(d_out, na * r)
    t, u = (x @ a.t()) * by, (dy @ b) * by
    out = {"dA": (u.t() @ x).reshape(na, r, d_in), "dB": (dy.t() @ t).reshape(d_out, na, r).permute(1, 0, 2).contiguous()}
    if c["dx"]:
        out["dX"] = (s["base"].float() + u @ a).to(s["base"].dtype)
    return out


def _plain_policy(s):
    c = s["case"]
    z = s["logits"].float() / c["temp"]
    n, v = z.shape
    m = z.amax(1, keepdim=True)
    e = torch.exp(z - m)
    total = e.sum(1, keepdim=True, dtype=torch.float64)
    t = s["targets"].long()[:, None]
    there = (t >= 0) & (t < v)
    at = t.clamp(0, v - 1)
    # the row's few numbers in 64 bits: a ratio next to the border, small differences of logarithms
    lp = (s["logits"].gather(1, at).double() / c["temp"] - m.double() - torch.log(total))[:, 0]
    a = s["advantage"].double()
    ratio = torch.exp(lp - s["old"].double())
    kept = ratio.clamp(1.0 - 0.2, 1.0 + 0.2)
    loss = -torch.minimum(ratio * a, kept * a)
    d_lp = torch.where(ratio * a <= kept * a, -ratio * a, torch.zeros_like(a))
    kl = torch.zeros_like(lp)
    if s["ref"] is not None:
        d = s["ref"].double() - lp
        kl = torch.expm1(d) - d
        loss = loss + c["kl"] * kl
        d_lp = d_lp - c["kl"] * torch.expm1(d)
    scored = there[:, 0]
    zero = torch.zeros((), dtype=torch.float64, device=z.device)
    out = {name: torch.where(scored, x, zero).float() for name, x in
           (("loss", loss), ("logprob", lp), ("ratio", ratio), ("kl", kl))}
    if c["grad"]:
        f = torch.where(scored, d_lp * s["weight"].double() / c["temp"], zero)
        g = e * (-f[:, None] / total).float()
        at_t = (-torch.expm1(lp) * f)[:, None].float()   # 1 - q without the difference
        g.scatter_(1, at, torch.where(there, at_t, torch.zeros_like(at_t)))
        out["grad"] = g.to(s["logits"].dtype)
    return out


# ---------------------------------------------------------------- one pass
def _run_own(s):
    from post_weight_quantization_08_amd import pipeline as P

    c, keep = s["case"], s["keep"]
    if c["op"] == "quantize":
        if not keep:
            keep["out"] = P.fp8_quantize_buffers(s["X"], tiles=c["tiles"])
        return P.fp8_quantize(s["X"], tiles=c["tiles"], **keep)
    if c["op"] == "matmul":
        scales = _scale_type(s["x_scales"]) if s["x_scales"] is not None else None
        if not keep:
            keep["Y"], keep["ws"] = P.fp8_matmul_buffers(s["X"], s["W"], y_dtype=_TYPES[c["y"]])
        return P.fp8_matmul(s["X"], s["W"], _scale_type(s["w_scales"]), x_scales=scales, **keep)
    if c["op"] == "grad":
        scales = _scale_type(s["x_scales"]) if s["x_scales"] is not None else None
        if not keep:
            keep["out"], keep["ws"] = P.lora_grad_buffers(s["X"], s["dY"], s["A"], s["B"],
                                                          dx_dtype=s["base"].dtype if c["dx"] else None)
        return P.lora_grad(s["X"], s["dY"], s["A"], s["B"], s["adapter"], s["scale"], x_scales=scales, base=s["base"],
                           **keep)
    if not keep:
        keep["out"], keep["ws"] = P.policy_loss_buffers(s["logits"], want_grad=c["grad"])
    return P.policy_loss(s["logits"], s["targets"], s["old"], s["advantage"], ref_logprob=s["ref"], clip_low=0.2,
                         clip_high=0.2, kl_coef=c["kl"], temperature=c["temp"], weight=s["weight"],
                         want_grad=c["grad"], **keep)


def run(state):
    if own:
        return _run_own(state)
    op = state["case"]["op"]
    if op == "quantize":
        return _plain_quantize(state)
    if op == "matmul":
        return _plain_matmul(state)
    if op == "grad":
        return _plain_grad(state)
    return _plain_policy(state)


_SIZE = {"f32": 4, "f16": 2, "bf16": 2, "e4m3": 1}


def work(case):
    if case["op"] == "quantize":
        cells = case["rows"] * case["cols"]
        return {"bytes": cells * (_SIZE[case["dtype"]] + (2 if case["tiles"] else 1)) + cells // _BLOCK, "flops": 3 * cells}
    if case["op"] == "matmul":
        m, k, n = case["m"], case["d_in"], case["d_out"]
        return {"bytes": m * k * _SIZE[case["x"]] + n * k + m * n * _SIZE[case["y"]], "flops": 2 * m * n * k}
    if case["op"] == "grad":
        m, d_in, d_out, r = case["m"], case["d_in"], case["d_out"], case["rank"]
        n = min(case["adapters"], m)
        b = m * d_in * _SIZE[case["x"]] + m * d_out * _SIZE[case["dy"]] + n * r * (d_in + d_out) * (2 + 4)
        b += 2 * m * d_in * 2 if case["dx"] else 0
        return {"bytes": b, "flops": 2 * m * r * (2 * d_in + 2 * d_out + (d_in if case["dx"] else 0))}
    cells = case["n"] * case["vocab"] * _SIZE[case["dtype"]]
    return {"bytes": cells * (2 if case["grad"] else 1) + case["n"] * 36,
            "flops": (6 if case["grad"] else 4) * case["n"] * case["vocab"]}


# ---------------------------------------------------------------- the definitions in 64 bits
def _power_of_two(e):
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _exact_scale(top):
    """The smallest power of two, at least 2^-100, that brings `top` to 448 or less."""
    _, e = torch.frexp(top.clamp(min=2.0 ** -130) / 448.0)
    s = _power_of_two(e - 1)
    s = torch.where(s * 448.0 >= top, s, 2.0 * s)
    return s.clamp(min=2.0 ** -100)


def _exact_codes(v):
    """Nearest value with four significant bits, of a multiple of 2^-9; ties to even."""
    _, e = torch.frexp(v)
    step = _power_of_two((e - 4).clamp(min=-9))
    return torch.round(v / step) * step


def _exact_rows(x):
    """(codes, scales) of rows in blocks, padded with zeros."""
    rows, cols = x.shape
    full = torch.zeros(rows, _padded(cols), dtype=torch.float64, device=x.device)
    full[:, :cols] = x.double()
    blocks = full.view(rows, -1, _BLOCK)
    s = _exact_scale(blocks.abs().amax(2))
    return _exact_codes(blocks / s[:, :, None]).reshape(rows, -1), s


def _exact_tiles(x):
    rows, cols = x.shape
    full = torch.zeros(_padded(rows), _padded(cols), dtype=torch.float64, device=x.device)
    full[:rows, :cols] = x.double()
    tiles = full.view(_padded(rows) // _BLOCK, _BLOCK, -1, _BLOCK)
    s = _exact_scale(tiles.abs().amax(3).amax(1))
    return _exact_codes(tiles / s[:, None, :, None]).reshape(full.shape), s


def _stands_for(codes, b, height):
    """Values of codes with scale bytes of blocks of `height` rows."""
    s = _power_of_two(b.to(torch.int64) - 127)
    s = s.repeat_interleave(_BLOCK, dim=1)
    if height > 1:
        s = s.repeat_interleave(height, dim=0)[:codes.shape[0]]
    return codes.float().double() * s


def _exact_policy_rows(s, w, c):
    x = s["logits"][w].double() / c["temp"]
    n, v = x.shape
    logq = torch.log_softmax(x, 1)
    t = s["targets"][w].long()
    there = (t >= 0) & (t < v)
    at = t.clamp(0, v - 1)[:, None]
    lp = logq.gather(1, at)[:, 0]
    a, old = s["advantage"][w].double(), s["old"][w].double()
    ratio = (lp - old).exp()
    inside_low, inside_high = ratio >= 0.8, ratio <= 1.2
    # the smaller of both products: outside the interval on the side where the advantage pulls, it is constant
    frozen = torch.where(a >= 0, ~inside_high, ~inside_low)
    border = torch.where(a >= 0, torch.full_like(a, 1.2), torch.full_like(a, 0.8))
    loss = torch.where(frozen, -border * a, -ratio * a)
    coef = torch.where(frozen, torch.zeros_like(a), -ratio * a)
    kl = torch.zeros_like(lp)
    if s["ref"] is not None:
        d = s["ref"][w].double() - lp
        kl = d.exp() - d - 1.0
        loss = loss + c["kl"] * kl
        coef = coef + c["kl"] * (1.0 - d.exp())
    on = there.double()
    out = [loss * on, lp * on, ratio * on, kl * on]
    if c["grad"]:
        f = (coef * s["weight"][w].double() * on / c["temp"])[:, None]
        g = logq.exp_().mul_(-f)
        g.scatter_add_(1, at, f)
        out.append(g)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "quantize":
        codes, scales = (_exact_tiles if case["tiles"] else _exact_rows)(s["X"])
        out = {"codes": codes[:case["rows"]], "scales": scales}
        if case["tiles"]:
            out["codes_t"] = codes.t()[:case["cols"]]
            out["scales_t"] = scales.t()
        return out
    if case["op"] == "matmul":
        w = _stands_for(s["W"], s["w_scales"], _BLOCK)
        if case["x"] == "e4m3":
            x = _stands_for(s["X"], s["x_scales"], 1)
        else:
            codes, scales = _exact_rows(s["X"])
            x = codes * scales.repeat_interleave(_BLOCK, dim=1)
        return x @ w.T
    if case["op"] == "grad":
        x = _stands_for(s["X"], s["x_scales"], 1)[:, :case["d_in"]] if case["x"] == "e4m3" else s["X"].double()
        dy = s["dY"].double()
        out = {"dA": torch.zeros(s["A"].shape, dtype=torch.float64, device=x.device),
               "dB": torch.zeros(s["B"].shape, dtype=torch.float64, device=x.device)}
        if case["dx"]:
            out["dX"] = s["base"].double()
        for i in range(case["adapters"]):
            rows = torch.nonzero(s["adapter"] == i)[:, 0]
            if len(rows):
                a, b, f = s["A"][i].double(), s["B"][i].double(), s["scale"][i].double()
                u = f * (dy[rows] @ b)
                out["dA"][i] = u.T @ x[rows]
                out["dB"][i] = f * (dy[rows].T @ (x[rows] @ a.T))
                if case["dx"]:
                    out["dX"][rows] += u @ a
        return out
    step = max(1, (1 << 25) // case["vocab"])
    parts = [_exact_policy_rows(s, slice(i, i + step), case) for i in range(0, case["n"], step)]
    cols = [torch.cat(p) for p in zip(*parts)]
    return dict(zip(("loss", "logprob", "ratio", "kl", "grad"), cols))
