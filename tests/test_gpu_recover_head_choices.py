"""The example's gradients: from the hidden states as they are, unless they are to be kept in 8 bits."""
import numpy as np
import pytest

from examples import recover_head

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("keep_8_bit", [False, True])
def test_gradients(keep_8_bit):
    """Against float64.  bf16 operands: what is left is fp32 sums of 256 and 300 terms, 2^-23 of the sum of magnitudes for
    each addition.  In 8 bits an element is off by half a step, 2^-4 of itself, and small ones of a block by 2^-10 of the
    smallest power of two above its largest / 448, 2^-17 of the largest."""
    import torch
    from post_weight_quantization_08_amd import pipeline as P
    M, d_in, d_out, r, n = 300, 256, 515, 16, 2
    gen = torch.Generator(device="cuda").manual_seed(1)
    X = torch.randn(M, d_in, generator=gen, device="cuda").bfloat16()
    A, B = (torch.randn(n, r, d_in, generator=gen, device="cuda") * 0.1).bfloat16(), torch.randn(n, d_out, r, generator=gen, device="cuda").bfloat16()
    g = torch.randn(M, d_out, generator=gen, device="cuda").bfloat16()
    adapter = (torch.arange(M, device="cuda") * 2 // M).int()
    dA, dB = recover_head.gradients(P.fp8_quantize(X) if keep_8_bit else X, A, B, adapter, torch.ones(n, device="cuda"), g)
    for i in range(n):
        rows = (adapter == i).nonzero()[:, 0]
        x, y, a, b = (v.double() for v in (X[rows], g[rows], A[i], B[i]))
        off = 2.0 ** -4 * x.abs() + 2.0 ** -17 * x.abs().amax(1, keepdim=True) if keep_8_bit else torch.zeros_like(x)
        u, t = y @ b, x @ a.t()
        sums = 2.0 ** -23 * (d_in + d_out + M + 64)
        bA = u.abs().t() @ off + sums * ((y.abs() @ b.abs()).t() @ (x.abs() + off))
        bB = y.abs().t() @ (off @ a.abs().t()) + sums * (y.abs().t() @ ((x.abs() + off) @ a.abs().t()))
        assert bool(((dA[i].double() - u.t() @ x).abs() <= bA).all())
        assert bool(((dB[i].double() - y.t() @ t).abs() <= bB).all())


def test_both_run():
    for keep in (False, True):
        r = recover_head.run(steps=3, hidden=256, vocab=1001, tokens=128, show=lambda s: None, keep_8_bit=keep)
        assert np.isfinite([r["first"], r["last"], r["with"], r["without"]]).all() and r["untouched"]
