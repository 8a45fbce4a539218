"""The answer-side entry points reject bad arguments before touching a GPU."""
import pytest

from tests.test_abi_cpu import G  # noqa: F401  (fixture)

FAKE = 0x10000
BIG = 1 << 40


def _lp(G, x=FAKE, dtype=2, n=4, V=1000, ld=None, t=FAKE, T=1.0, k=5, lp=FAKE, lse=FAKE, ent=FAKE, tl=FAKE, ti=FAKE,
        ws=FAKE, ws_bytes=BIG):
    return G.lib.gptq_token_logprobs(x, dtype, n, V, V if ld is None else ld, t, T, k, lp, lse, ent, tl, ti, ws, ws_bytes, None)


def test_logprobs_argument_errors(G):
    E = G.EINVAL
    assert _lp(G, x=None) == E
    assert _lp(G, dtype=3) == E
    assert _lp(G, n=-1) == E
    assert _lp(G, V=0) == E
    assert _lp(G, V=1 << 31) == E
    assert _lp(G, ld=999) == E
    assert _lp(G, t=None) == E                      # a log probability needs its target
    for T in (0.0, -1.0, float("nan"), float("inf"), 1e-6):
        assert _lp(G, T=T) == E
    assert _lp(G, k=-1) == E
    assert _lp(G, k=6, V=5) == E
    assert _lp(G, tl=None) == E
    assert _lp(G, ti=None) == E
    assert _lp(G, k=0, lp=None, lse=None, ent=None) == E   # nothing asked
    assert _lp(G, x=FAKE + 1) == E
    assert _lp(G, x=FAKE + 2, dtype=0) == E
    assert _lp(G, k=129) == G.EUNSUPPORTED
    assert _lp(G, n=0) == G.OK
    need = G.gptq_workspace_size(G.OP_LOGPROBS, None, 1, 131072, 1, 20)
    if need:
        assert _lp(G, n=1, V=131072, k=20, ws_bytes=need - 1) == G.ENOMEM
        assert _lp(G, n=1, V=131072, k=20, ws=None) == G.ENOMEM


def _ds(G, x=FAKE, dtype=2, n=4, V=1000, ld=None, ids=FAKE, lp=FAKE, k=5, T=1.0, tail=1, w=None, loss=FAKE,
        grad=4 * FAKE, ld_g=None, ws=FAKE, ws_bytes=BIG):
    return G.lib.gptq_distill_topk(x, dtype, n, V, V if ld is None else ld, ids, lp, k, T, tail, w, loss, grad,
                                   V if ld_g is None else ld_g, ws, ws_bytes, None)


def test_distill_argument_errors(G):
    E = G.EINVAL
    assert _ds(G, x=None) == E
    assert _ds(G, dtype=-1) == E
    assert _ds(G, n=-1) == E
    assert _ds(G, V=0) == E
    assert _ds(G, ld=999) == E
    assert _ds(G, ids=None) == E
    assert _ds(G, lp=None) == E
    assert _ds(G, k=0) == E
    assert _ds(G, T=float("nan")) == E
    assert _ds(G, tail=2) == E
    assert _ds(G, loss=None, grad=None) == E
    assert _ds(G, ld_g=999) == E
    assert _ds(G, grad=FAKE, ld=1000, ld_g=1001) == E      # in place needs one stride
    assert _ds(G, grad=4 * FAKE + 1) == E
    assert _ds(G, k=129) == G.EUNSUPPORTED
    assert _ds(G, n=0) == G.OK
    need = G.gptq_workspace_size(G.OP_DISTILL, None, 1, 131072, 1, 20)
    if need:
        assert _ds(G, n=1, V=131072, k=20, ws_bytes=need - 1) == G.ENOMEM


def _lo(G, X=FAKE, dtype=2, M=4, d_in=256, ld_x=None, A=FAKE, B=FAKE, n=2, r=8, s=None, ad=FAKE, base=None, ld_b=0,
        Y=FAKE, ydt=0, d_out=96, ld_y=None, ws=FAKE, ws_bytes=BIG):
    return G.lib.gptq_lora_add(X, dtype, M, d_in, d_in if ld_x is None else ld_x, A, B, n, r, s, ad, base, ld_b, Y, ydt,
                               d_out, d_out if ld_y is None else ld_y, ws, ws_bytes, None)


def test_lora_argument_errors(G):
    E = G.EINVAL
    assert _lo(G, dtype=0) == E
    assert _lo(G, ydt=1) == E                       # bf16 rows into fp16
    assert _lo(G, M=-1) == E
    assert _lo(G, d_in=0) == E
    assert _lo(G, ld_x=255) == E
    assert _lo(G, ld_y=95) == E
    assert _lo(G, base=FAKE * 2, ld_b=95) == E
    assert _lo(G, base=FAKE, Y=FAKE, ld_b=100) == E
    assert _lo(G, n=0) == E
    assert _lo(G, r=0) == E
    for name in ("X", "A", "B", "ad", "Y"):
        assert _lo(G, **{name: None}) == E
    assert _lo(G, X=FAKE + 1) == E
    assert _lo(G, Y=FAKE + 2) == E                  # fp32 rows
    assert _lo(G, ws=FAKE + 16) == E
    assert _lo(G, r=129) == G.EUNSUPPORTED
    assert _lo(G, ws=None) == G.ENOMEM
    assert _lo(G, ws_bytes=G.gptq_workspace_size(G.OP_LORA, None, 96, 256, 4, 8) - 1) == G.ENOMEM
    assert _lo(G, M=0) == G.OK


def _wl(G, M=4, d_in=256, d_out=96, g=128, dtype=2, qw=FAKE, A=FAKE, n=2, r=8, ad=FAKE, ld_y=None, ws=FAKE, ws_bytes=BIG):
    return G.lib.gptq_w4a16_lora_matmul(FAKE, dtype, M, d_in, d_in, qw, FAKE, FAKE, None, d_out, g, A, FAKE, n, r, None,
                                        ad, FAKE, d_out if ld_y is None else ld_y, ws, ws_bytes, None)


def test_w4a16_lora_argument_errors(G):
    E = G.EINVAL
    assert _wl(G, dtype=0) == E
    assert _wl(G, M=0) == E
    assert _wl(G, d_in=200) == E
    assert _wl(G, A=None) == E
    assert _wl(G, ad=None) == E
    assert _wl(G, n=0) == E
    assert _wl(G, r=0) == E
    assert _wl(G, qw=FAKE + 8) == E
    assert _wl(G, ld_y=95) == E
    assert _wl(G, ws=FAKE + 16) == E
    assert _wl(G, M=65) == G.EUNSUPPORTED
    assert _wl(G, g=64) == G.EUNSUPPORTED
    assert _wl(G, r=129) == G.EUNSUPPORTED
    assert _wl(G, ws=None) == G.ENOMEM
    need = G.gptq_workspace_size(G.OP_W4A16_LORA, None, 96, 256, 4, 8)
    assert _wl(G, ws_bytes=need - 1) == G.ENOMEM


def test_workspace_of_the_answer_side_operators(G):
    for op in (G.OP_LOGPROBS, G.OP_DISTILL, G.OP_LORA, G.OP_W4A16_LORA):
        assert G.gptq_workspace_size(op, None, 64, 1024, 3, 16) >= 0
        with pytest.raises(G.GptqError):
            G.gptq_workspace_size(op, None, 64, 0, 3, 16)
        with pytest.raises(G.GptqError):
            G.gptq_workspace_size(op, None, 64, 1024, -1, 16)
    assert G.gptq_workspace_size(G.OP_LORA, None, 64, 1024, 64, 16) > 0
