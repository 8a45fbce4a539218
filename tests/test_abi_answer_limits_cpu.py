"""Limits of the answer-side entry points that are met before a GPU is."""
from tests.test_abi_cpu import G  # noqa: F401  (fixture)

FAKE = 0x10000


def test_rows_that_no_launch_can_hold_are_refused(G):
    """A workgroup of 256 threads per row, and a launch has fewer than 2^32 threads."""
    def call(n):
        return G.lib.gptq_token_logprobs(FAKE, 2, n, 1, 1, FAKE, 1.0, 1, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 1 << 40, None)
    assert call(1 << 24) == G.EINVAL
    assert call((1 << 24) + 1) == G.EINVAL
    assert call(0) == G.OK
