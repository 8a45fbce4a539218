"""Which calls of few tokens take one launch: those that need no workspace."""
import pytest

from tests.test_abi_cpu import G  # noqa: F401  (fixture)


@pytest.mark.parametrize("M,d_in,d_out,one", [
    (1, 128, 16, True), (16, 28672, 4096, True), (17, 128, 16, False), (1, 65536, 8192, True), (16, 4096, 8192, True),
    (8, 8192, 8192, True), (16, 8192, 8192, False), (9, 8192, 4097, False), (16, 4097, 8192, False), (1, 128, 8193, False)])
def test_one_launch(G, M, d_in, d_out, one):
    assert (G.gptq_workspace_size(G.OP_FP8_MATMUL, None, d_out, d_in, M, 1) == 0) == one
