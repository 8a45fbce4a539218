"""Quantizing to 8 bits refuses what no launch holds: 2^32 threads, 256 for every 64 blocks."""
from tests.test_abi_cpu import G  # noqa: F401  (fixture)
from tests.test_abi_fp8_cpu import FAKE, _m, _q

MOST = (1 << 30) - 64


def test_rows_of_one_column(G):
    for rows in (MOST + 1, (1 << 30) - 1, 1 << 30):
        assert _q(G, rows=rows, cols=1, ld_c=128) == G.EUNSUPPORTED
    assert _q(G, rows=MOST, cols=1, ld_c=128, X=None) == G.EINVAL      # taken, but for the pointer
    assert _q(G, rows=MOST // 2, cols=129, X=None) == G.EINVAL
    assert _q(G, rows=MOST // 2 + 1, cols=129) == G.EUNSUPPORTED


def test_products_that_quantize_their_tokens(G):
    for M, d_in in ((1 << 22, 1 << 15), (1 << 22, 1 << 22)):
        assert _m(G, M=M, d_in=d_in, ld_w=d_in, work_bytes=1 << 62) == G.EUNSUPPORTED
        assert _m(G, dtype=3, xs=FAKE, M=M, d_in=d_in, ld_w=d_in, Y=None) == G.EINVAL      # codes are there already
