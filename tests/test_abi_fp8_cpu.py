"""The 8-bit entry points reject bad arguments before touching a GPU."""
import pytest

from tests.test_abi_cpu import G  # noqa: F401  (fixture)

FAKE = 0x10000
BIG = 1 << 40


def _q(G, X=FAKE, dtype=2, rows=4, cols=200, ld_x=None, block=1, codes=FAKE, ld_c=256, scales=FAKE, codes_t=None,
       ld_ct=0, scales_t=None):
    return G.lib.gptq_fp8_quantize(X, dtype, rows, cols, cols if ld_x is None else ld_x, block, codes, ld_c, scales,
                                   codes_t, ld_ct, scales_t, None)


def test_quantize_argument_errors(G):
    E = G.EINVAL
    for dtype in (-1, 3, 4):
        assert _q(G, dtype=dtype) == E
    assert _q(G, rows=-1) == E
    assert _q(G, cols=0) == E
    assert _q(G, ld_x=199) == E
    assert _q(G, block=64) == E
    assert _q(G, ld_c=208) == E                    # not whole blocks
    assert _q(G, ld_c=264) == E                    # not on 16 bytes
    for name in ("X", "codes", "scales"):
        assert _q(G, **{name: None}) == E
    assert _q(G, X=FAKE + 1) == E
    assert _q(G, X=FAKE + 2, dtype=0) == E
    assert _q(G, codes=FAKE + 8) == E
    turn = dict(block=128, codes_t=FAKE, ld_ct=128, scales_t=FAKE)
    assert _q(G, **dict(turn, block=1)) == E       # rows have no transpose
    assert _q(G, **dict(turn, scales_t=None)) == E
    assert _q(G, **dict(turn, codes_t=None)) == E
    assert _q(G, **dict(turn, ld_ct=112)) == E
    assert _q(G, **dict(turn, codes_t=FAKE + 8)) == E
    assert _q(G, rows=1 << 28, cols=1024, ld_c=1024) == G.EUNSUPPORTED
    assert _q(G, rows=0) == G.OK
    assert _q(G, **dict(turn, rows=0)) == G.OK


def _m(G, X=FAKE, dtype=2, xs=None, M=4, d_in=256, ld_x=None, W=FAKE, ld_w=256, ws=FAKE, d_out=96, Y=FAKE, ydt=0,
       ld_y=None, work=FAKE, work_bytes=BIG):
    return G.lib.gptq_fp8_matmul(X, dtype, xs, M, d_in, d_in if ld_x is None else ld_x, W, ld_w, ws, d_out, Y, ydt,
                                 d_out if ld_y is None else ld_y, work, work_bytes, None)


def test_matmul_argument_errors(G):
    E = G.EINVAL
    for dtype in (-1, 4):
        assert _m(G, dtype=dtype) == E
    for dtype in (-1, 3):
        assert _m(G, ydt=dtype) == E
    assert _m(G, M=-1) == E
    assert _m(G, d_in=0, ld_x=1) == E
    assert _m(G, d_out=0) == E
    assert _m(G, ld_x=255) == E
    assert _m(G, ld_y=95) == E
    assert _m(G, ld_w=240) == E
    assert _m(G, d_in=200, ld_w=208) == E          # rows of weights are whole blocks
    assert _m(G, ld_w=264) == E
    for name in ("X", "W", "ws", "Y"):
        assert _m(G, **{name: None}) == E
    codes = dict(dtype=3, xs=FAKE)
    assert _m(G, **dict(codes, xs=None)) == E
    assert _m(G, **dict(codes, d_in=200)) == E     # codes come in whole blocks
    assert _m(G, **dict(codes, ld_x=264)) == E
    assert _m(G, **dict(codes, X=FAKE + 8)) == E
    assert _m(G, W=FAKE + 8) == E
    assert _m(G, Y=FAKE + 2) == E
    assert _m(G, X=FAKE + 1) == E
    assert _m(G, work=FAKE + 16) == E
    for big in (dict(M=1 << 23), dict(d_in=1 << 23, ld_w=1 << 23), dict(d_out=1 << 23)):
        assert _m(G, **big) == G.EUNSUPPORTED
    assert _m(G, M=0) == G.OK
    for sizes in (dict(M=300), dict(M=100, d_in=4096, ld_w=4096)):
        need = G.gptq_workspace_size(G.OP_FP8_MATMUL, None, 96, sizes.get("d_in", 256), sizes["M"], 1)
        assert need > 0
        assert _m(G, **sizes, work_bytes=need - 1) == G.ENOMEM
        assert _m(G, **sizes, work=None) == G.ENOMEM


def test_workspace(G):
    assert G.gptq_workspace_size(G.OP_FP8_MATMUL, None, 96, 256, 0, 1) == 0
    for bad in (dict(d_in=0), dict(d_out=0), dict(n_rows=-1)):
        with pytest.raises(G.GptqError):
            G.gptq_workspace_size(G.OP_FP8_MATMUL, None, **dict(dict(d_out=96, d_in=256, n_rows=4, batch=1), **bad))


def test_wrappers_refuse_cpu_tensors(G):
    import torch
    from post_weight_quantization_08_amd import pipeline as P
    x = torch.zeros(4, 256)
    w = torch.zeros(96, 256).to(torch.float8_e4m3fn)
    with pytest.raises(ValueError):
        P.fp8_quantize(x)
    with pytest.raises(ValueError):
        P.fp8_matmul(x, w, torch.zeros(1, 2, dtype=torch.uint8).view(torch.float8_e8m0fnu))
