"""The 4-bit projection's kernel for many outputs, without and with adapters,
for every number of token tiles and of waves per workgroup it is built for, and
both kernels on each side of the rule between them."""
import numpy as np
import pytest

import oracle as O
import synth
from tests import answer_data as D
from tests.gpu_run import log
from tests.parity import w4a16_error_bound

pytestmark = pytest.mark.gpu

# (d_out, d_in, M, g, type, act-order, rank, adapters)
CASES = [
    # a tile of tokens: 4, 5, 6, 7 and 8 waves, two rounds, ragged rows
    (12288, 128, 12, 128, "bf16", False, 16, 3),
    (13001, 640, 7, 128, "f16", True, 8, 5),
    (20480, 384, 16, 128, "bf16", False, 33, 4),
    (24500, 256, 9, 256, "f16", False, 16, 9),
    (28672, 2048, 5, 128, "bf16", True, 16, 5),
    (32003, 640, 8, 128, "bf16", False, 4, 3),
    (40007, 384, 13, 128, "f16", False, 64, 13),
    # two tiles
    (8192, 512, 32, 128, "bf16", True, 16, 7),
    (8704, 640, 17, 128, "f16", False, 32, 3),
    (20011, 512, 24, 128, "bf16", False, 128, 2),
    (28672, 896, 29, 128, "f16", True, 16, 29),
    # three
    (8200, 256, 33, 128, "bf16", False, 16, 5),
    (19001, 640, 40, 128, "f16", False, 24, 40),
    (28683, 384, 48, 128, "bf16", True, 8, 6),
    # four
    (12288, 256, 64, 256, "f16", False, 64, 64),
    (20480, 640, 49, 128, "bf16", True, 16, 3),
    (30001, 512, 60, 128, "bf16", False, 100, 2),
    # the other kernel, next to the rule's edges
    (8192, 512, 31, 128, "bf16", False, 16, 3),
    (12288, 640, 11, 128, "f16", True, 16, 3),
    (13001, 640, 6, 128, "bf16", False, 16, 3),
    (12288, 384, 20, 128, "bf16", False, 16, 3),
    (12288, 128, 50, 128, "f16", False, 16, 3),
]


@pytest.mark.parametrize("d_out,d_in,m,g,xdt,act_order,rank,n", CASES)
def test_both_kernels_give_the_same_sums(d_out, d_in, m, g, xdt, act_order, rank, n):
    """Slices of 4000 outputs at a time always take the kernel for few: equal bit by bit, and some rows of the
    outputs against the oracle."""
    import torch
    from post_weight_quantization_08_amd import pipeline as P

    i = CASES.index((d_out, d_in, m, g, xdt, act_order, rank, n))
    cfg = synth.CONFIGS["up_proj_70b"].scaled(f"w4wide2:{i}", 700 + i, d_out=d_out, d_in=d_in, group_size=g, x_dtype=xdt)
    codes, scales, zeros, perm, g_idx = synth.w4_layer(cfg, act_order, 0)
    Xs, As, Bs, s = D.adapters(m, d_in, d_out, rank, n, xdt, 41)
    a = np.random.default_rng([105, i]).integers(-1, n + 1, m).astype(np.int32)
    X, A, B = (D.to_torch(t, xdt) for t in (Xs, As, Bs))
    ad, sd = torch.from_numpy(a).cuda(), torch.from_numpy(s).cuda()
    cd = torch.from_numpy(codes).cuda()
    pd = torch.from_numpy(perm).cuda() if perm is not None else None
    qw = P.pack_int4_permuted(cd, pd) if pd is not None else P.pack(cd, 4)
    sc, zd = torch.from_numpy(scales.view(np.int16)).cuda(), torch.from_numpy(zeros).cuda()
    plain = P.w4a16_matmul(X, qw, sc, zd, g, perm=pd)
    Y = P.w4a16_lora_matmul(X, qw, sc, zd, g, A, B, ad, sd, perm=pd)
    for o in range(0, d_out, 4000):
        e = min(o + 4000, d_out)
        assert torch.equal(P.w4a16_matmul(X, qw[o:e], sc[o:e], zd[o:e], g, perm=pd), plain[:, o:e])
        assert torch.equal(P.w4a16_lora_matmul(X, qw[o:e], sc[o:e], zd[o:e], g, A, B[:, o:e].contiguous(), ad, sd, perm=pd),
                           Y[:, o:e])
    none = torch.from_numpy((a < 0) | (a >= n)).cuda()
    assert torch.equal(plain[none], Y[none])
    rows = np.unique(np.concatenate([[0, d_out - 1], np.random.default_rng(i).integers(0, d_out, 300)]))
    Xf, Af, Bf = D.exact(Xs, xdt), D.exact(As, xdt), D.exact(Bs[:, rows], xdt)
    s32 = scales[rows].view(np.float16).astype(np.float32)
    base = O.w4a16_matmul(Xf, O.pack_int4(codes[rows]), s32, zeros[rows], g_idx)
    tol = w4a16_error_bound(Xf, codes[rows], s32, zeros[rows], g_idx, bias=128.0 if xdt == "bf16" else 0.0)
    err = np.abs(plain.double().cpu().numpy()[:, rows] - base)
    assert np.all(err <= tol), float(np.max(err / tol))
    want = O.lora(Xf, Af, Bf, a, s, base)
    tol = tol + D.lora_bound(Xf, Af, Bf, a, s, want, xdt, "f32")
    err = np.abs(Y.double().cpu().numpy()[:, rows] - want)
    log(f"[gpu] w4a16 wide {d_out}x{d_in} M={m} {xdt} r={rank}: worst error / bound {np.max(err / tol):.3f}")
    assert np.all(err <= tol)
