"""Gradients of adapters through the loops of long sums, and the 24 bits that U, T and fp32 dY keep.

Loops: operands are small whole numbers and scales powers of two, so that U, T and every partial sum are numbers that fp32
holds: the results are equal to the definition's, dX rounded once.

Digits: one token per adapter and factors with a single 1, so that U and T are known products.  A 24-bit number is three bf16
terms without a rest; of the products of terms those of an order below 2^-24 are left out (below 2^-25 together); U and T are
rounded once, and at most eight additions follow, each off by a step (2^-23) at most: 10 steps in all."""
import numpy as np
import pytest

from oracle import fp8 as F8

pytestmark = pytest.mark.gpu
STEP = 2.0 ** -23


def torch_type(name):
    import torch
    return {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[name]


def mix(M, n, kind, gen):
    import torch
    if kind == "one":
        return torch.zeros(M, dtype=torch.int32, device="cuda")
    if kind == "turns":                                   # a wave's 32 tokens have one adapter, a workgroup's several
        return ((torch.arange(M, device="cuda") + 16) // 32 % (n + 1) - 1).int()
    if kind == "any":
        return torch.randint(-1, n + 1, (M,), generator=gen, device="cuda").int()
    cut = torch.sort(torch.randint(0, M, (2 * n,), generator=gen, device="cuda")).values
    a = torch.searchsorted(cut, torch.arange(M, device="cuda"), right=True)
    return torch.where(a == 1, -1, a % n).int()


# (M, d_in, d_out, rank, adapters, factors, X, dY, mix, dX).  A part of the first sums has 5 to 24 blocks (odd and even
# numbers, the last one whole or not), a chunk 3 to 16 steps, a workgroup of dX 7 to 25 tiles of tokens or more, of one
# adapter and of several
CASES = [
    (8192, 3000, 2500, 16, 3, "bf16", "bf16", "bf16", "runs", "bf16"),
    (8192, 3000, 2500, 64, 1, "bf16", "e4m3", "f32", "one", "bf16"),
    (8192, 3000, 2500, 16, 1, "f16", "f16", "f16", "one", "f16"),
    (8192, 2944, 2560, 32, 2, "f16", "e4m3", "f16", "runs", "f32"),
    (5000, 2990, 2501, 100, 2, "f16", "f16", "f32", "runs", "f32"),
    (8000, 2900, 1030, 128, 2, "bf16", "e4m3", "bf16", "runs", "bf16"),
    (8192, 11008, 300, 32, 1, "bf16", "e4m3", "bf16", "one", "bf16"),
    (8192, 300, 4096, 64, 4, "bf16", "bf16", "f32", "runs", "f32"),
    (4096, 6000, 5000, 24, 5, "f16", "e4m3", "f16", "any", "f16"),
    (4096, 1300, 1290, 10, 40, "bf16", "bf16", "f32", "any", "bf16"),
    (2048, 9000, 9001, 8, 1, "bf16", "bf16", "bf16", "one", "f32"),
    (1200, 5762, 286, 48, 3, "f16", "f16", "f32", "runs", None),
    (20000, 700, 520, 4, 7, "f16", "e4m3", "f32", "runs", "f16"),
    (3000, 3000, 2500, 64, 6, "bf16", "e4m3", "f32", "turns", "bf16"),
    (2048, 4100, 4001, 16, 3, "f16", "f16", "f16", "turns", None),
    (40, 28672, 14336, 16, 2, "bf16", "bf16", "f32", "any", "bf16"),
]


@pytest.mark.parametrize("M,d_in,d_out,rank,n,ft,xt,yt,kind,dxt", CASES)
def test_sums_that_fp32_holds_are_exact(M, d_in, d_out, rank, n, ft, xt, yt, kind, dxt):
    import torch
    from post_weight_quantization_08_amd import pipeline as P
    gen = torch.Generator(device="cuda").manual_seed(M + d_in + rank)

    def whole(shape, most, share=1.0):
        x = torch.randint(-most, most + 1, shape, generator=gen, device="cuda").float()
        return x * (torch.rand(shape, generator=gen, device="cuda") < share)
    # few of each, so that no sum of magnitudes leaves the 24 bits (asserted below)
    x, dy = whole((M, d_in), 2, 0.5), whole((M, d_out), 2, 0.5)
    a, b = whole((n, rank, d_in), 1, 0.1), whole((n, d_out, rank), 1, 0.1)
    scale = 2.0 ** torch.randint(-1, 2, (n,), generator=gen, device="cuda").float()
    adapter = mix(M, n, kind, gen)
    base = whole((M, d_in), 8) if dxt else None
    kw = {}
    if xt == "e4m3":
        q = P.fp8_quantize(x)
        X, kw["x_scales"] = q["codes"], q["scales"]
    else:
        X = x.to(torch_type(xt))
    dY, A, B = dy.to(torch_type(yt)), a.to(torch_type(ft)), b.to(torch_type(ft))
    got = P.lora_grad(X, dY, A, B, adapter, scale, base=base.to(torch_type(dxt)) if dxt else None, **kw)
    assert ("dX" in got) == (dxt is not None)
    dX = base.double() if dxt else None
    for i in range(n):
        rows = torch.nonzero(adapter == i)[:, 0]
        xi, yi, s = x[rows].double(), dy[rows].double(), float(scale[i])
        u, t = s * (yi @ b[i].double()), s * (xi @ a[i].double().t())
        # multiples of a half; sums of magnitudes below 2^23
        assert float((u.abs().t() @ xi.abs()).max() if len(rows) else 0) < 2 ** 23
        assert float((yi.abs().t() @ t.abs()).max() if len(rows) else 0) < 2 ** 23
        for name, want in (("dA", u.t() @ xi), ("dB", yi.t() @ t)):
            bad = got[name][i].double() != want
            assert not bool(bad.any()), (name, i, int(bad.sum()), bad.nonzero()[:4].tolist())
        if dxt:
            dX[rows] += u @ a[i].double()
    if dxt:
        bad = got["dX"] != dX.float().to(torch_type(dxt))
        assert not bool(bad.any()), ("dX", int(bad.sum()), bad.nonzero()[:4].tolist())


def bf16_terms(v, n):
    """The first n bf16 terms' sum of float32 values."""
    out, left = np.zeros_like(v, dtype=np.float64), v.astype(np.float32)
    for _ in range(n):
        w = left.view(np.uint32).astype(np.uint64)
        t = ((w + 0x7FFF + ((w >> 16) & 1)) >> 16 << 16).astype(np.uint32).view(np.float32)
        out += t
        left = left - t
    return out


@pytest.mark.parametrize("ft,xt,yt", [("bf16", "bf16", "bf16"), ("bf16", "bf16", "f32"), ("f16", "f16", "f16"),
                                      ("f16", "f16", "f32"), ("bf16", "e4m3", "f32"), ("f16", "e4m3", "f16")])
@pytest.mark.parametrize("rank", [8, 40, 100])
def test_u_t_and_wide_gradients_keep_24_bits(rank, ft, xt, yt):
    import torch
    from post_weight_quantization_08_amd import pipeline as P
    n, d_in, d_out = 300, 200, 144
    r = np.random.default_rng([9, rank])

    def stored(v, kind):
        return torch.from_numpy(v.astype(np.float32)).to(torch_type(kind)).double().numpy()
    x = r.standard_normal((n, d_in))
    if xt == "e4m3":
        c, b = F8.fp8_quantize(x.astype(np.float32).astype(np.float64))
        x = F8.fp8_values(c, b)[:, :d_in]
        X, kw = torch.from_numpy(c).cuda().view(torch.float8_e4m3fn), {"x_scales": torch.from_numpy(b).cuda().view(torch.float8_e8m0fnu)}
    else:
        x = stored(x, xt)
        X, kw = torch.from_numpy(x).float().to(torch_type(xt)).cuda(), {}
    dy = stored(r.standard_normal((n, d_out)), yt)
    scale = r.uniform(0.5, 2, n).astype(np.float32)
    # rank j reads element i_j of a token and column o_j of its gradient
    at_i = np.stack([r.permutation(d_in)[:rank] for _ in range(n)])
    at_o = np.stack([r.permutation(d_out)[:rank] for _ in range(n)])
    A, B = np.zeros((n, rank, d_in)), np.zeros((n, d_out, rank))
    A[np.arange(n)[:, None], np.arange(rank), at_i] = 1
    B[np.arange(n)[:, None], at_o, np.arange(rank)] = 1
    adapter = r.permutation(n)
    dev = [torch.from_numpy(v).float().cuda() for v in (dy, A, B)]
    out = {"dA": torch.empty(n, rank, d_in, device="cuda"), "dB": torch.empty(n, d_out, rank, device="cuda"),
           "dX": torch.empty(n, d_in, device="cuda")}
    P.lora_grad(X, dev[0].to(torch_type(yt)), dev[1].to(torch_type(ft)), dev[2].to(torch_type(ft)),
                torch.from_numpy(adapter.astype(np.int32)).cuda(), torch.from_numpy(scale).cuda(), out=out, **kw)
    got = {k: v.double().cpu().numpy() for k, v in out.items()}
    lost = {"dA": 0.0, "dB": 0.0, "dX": 0.0}
    for m in range(n):
        a, s = adapter[m], float(scale[adapter[m]])
        u, t = s * dy[m, at_o[a]], s * x[m, at_i[a]]
        u2, t2 = bf16_terms(u.astype(np.float32), 2), bf16_terms(t.astype(np.float32), 2)
        want = {"dA": np.outer(u, x[m]), "dB": np.outer(dy[m], t), "dX": np.zeros(d_in)}
        fewer = {"dA": np.outer(u2, x[m]), "dB": np.outer(dy[m], t2), "dX": np.zeros(d_in)}
        want["dX"][at_i[a]], fewer["dX"][at_i[a]] = u, u2
        for k in want:
            have = got[k][m] if k == "dX" else got[k][a]
            err = np.abs(have - want[k])
            assert np.all(err <= 10 * STEP * np.abs(want[k])), (k, m, float((err / np.maximum(np.abs(want[k]), 1e-300)).max()))
            nz = want[k] != 0
            lost[k] = max(lost[k], float((np.abs(fewer[k] - want[k])[nz] / np.abs(want[k][nz])).max()))
    # two terms of U and T would not pass
    assert min(lost.values()) > 20 * STEP, lost
