"""8-bit products through the loops of long sums, in every kernel and output type.

Operands are small whole numbers as codes, with power-of-two scales that change from block to block: every product and
every partial sum is a number that fp32 holds (a multiple of 2^-4 below 2^20), and no product is 2^-13 of another.  Whatever
the order of the sum, the result is exact, and an output is it rounded once: results are equal, bit for bit."""
import numpy as np
import pytest

from oracle import fp8 as F

pytestmark = pytest.mark.gpu


def kernel_of(M, d_in, d_out):
    """Which kernel takes these sizes: few tokens, or tiles of so many tokens."""
    if M <= 16 and (d_out <= 4096 or d_out <= 8192 and M * d_in <= 1 << 16):
        return "few"
    if M > 128 and -(-M // 256) * -(-d_out // 256) >= 256:
        return 256
    if M <= 32:
        return 32
    return 64 if M <= 64 or -(-M // 128) * -(-d_out // 128) < 512 else 128


def codes(rows, cols, height, gen):
    """(codes, scale bytes, values in fp32) of 0, 1, 2 and 3, either sign; scales from 2^-2 to 2^2."""
    import torch
    table = torch.tensor([0x00, 0x38, 0x40, 0x44, 0xB8, 0xC0, 0xC4], dtype=torch.uint8, device="cuda")
    nb = -(-cols // 128)
    c = table[torch.randint(0, 7, (rows, nb * 128), generator=gen, device="cuda")]
    c[:, cols:] = 0
    b = torch.randint(125, 130, (-(-rows // height), nb), generator=gen, device="cuda").to(torch.uint8)
    value = torch.from_numpy(F.e4m3_values(np.arange(256))).float().cuda()[c.int()]
    scale = torch.exp2(b.float() - 127).repeat_interleave(height, 0)[:rows].repeat_interleave(128, 1)
    return c.view(torch.float8_e4m3fn), b.view(torch.float8_e8m0fnu), value * scale


def product(x, w):
    """In float64, the sum in slices."""
    import torch
    y = torch.zeros(x.shape[0], w.shape[0], dtype=torch.float64, device="cuda")
    for k in range(0, x.shape[1], 4096):
        y += x[:, k:k + 4096].double() @ w[:, k:k + 4096].double().t()
    return y


def compare(Y, want, what):
    import torch
    rounded = want.float().to(Y.dtype)
    assert torch.equal(want.float().double(), want) and bool(torch.isfinite(rounded).all()), what
    bad = Y != rounded
    assert not bool(bad.any()), (what, bad.nonzero()[:4].tolist(), Y[bad][:4].tolist(), rounded[bad][:4].tolist())


# (M, d_in, d_out, outputs, kernel).  Tiles of 256: odd and even numbers of blocks, words of scales that end inside four
# blocks, one word more than is kept at a time (120 blocks), twice that; the others: sums longer than any listed width
CASES = [
    (4100, 384, 4099, "bf16", 256), (4100, 640, 4099, "f16", 256), (4100, 1152, 4099, "bf16", 256),
    (4100, 1536, 4099, "f16", 256), (2100, 15360, 8200, "bf16", 256), (2100, 15488, 8200, "f16", 256),
    (2100, 15616, 8200, "bf16", 256), (2100, 31104, 8200, "bf16", 256), (65600, 128, 250, "bf16", 256),
    (2100, 1664, 8200, "f32", 256),
    (1100, 384, 7300, "bf16", 128), (1100, 1152, 7300, "f16", 128), (1111, 15488, 7301, "bf16", 128),
    (1100, 1024, 7300, "f32", 128),
    (65, 28672, 1000, "bf16", 64), (300, 14336, 2000, "f16", 64), (777, 11008, 4001, "f32", 64), (48, 28672, 515, "f32", 64),
    (17, 28672, 1000, "f16", 32), (32, 14336, 8200, "bf16", 32), (5, 28672, 9000, "f32", 32),
    (1, 28672, 1000, "bf16", "few"), (16, 14336, 515, "f16", "few"), (7, 15488, 130, "f32", "few"),
]


@pytest.mark.parametrize("M,d_in,d_out,yt,kernel", CASES)
def test_sums_that_fp32_holds_are_exact(M, d_in, d_out, yt, kernel):
    import torch
    from post_weight_quantization_08_amd import pipeline as P
    assert kernel_of(M, d_in, d_out) == kernel
    gen = torch.Generator(device="cuda").manual_seed(M + d_in)
    X, xs, x = codes(M, d_in, 1, gen)
    W, ws, w = codes(d_out, d_in, 128, gen)
    dt = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[yt]
    want = product(x, w)
    Y = P.fp8_matmul(X, W, ws, x_scales=xs, y_dtype=dt)
    compare(Y, want, f"{M}x{d_in}x{d_out} codes {yt}")
    # the values themselves, quantized by the call: other codes of the same numbers
    Y.fill_(9)
    P.fp8_matmul(x.bfloat16(), W, ws, Y=Y)
    compare(Y, want, f"{M}x{d_in}x{d_out} values {yt}")


def test_rows_far_apart():
    """Row strides above 2^23: tiles of 256 by the kernel that takes any stride."""
    import torch
    from post_weight_quantization_08_amd import pipeline as P
    M, d_in, d_out, ld = 130, 640, 65600, (1 << 23) + 16
    assert kernel_of(M, d_in, d_out) == 256
    gen = torch.Generator(device="cuda").manual_seed(5)
    X, xs, x = codes(M, d_in, 1, gen)
    W, ws, w = codes(d_out, d_in, 128, gen)
    far = torch.empty(M * ld, dtype=torch.uint8, device="cuda").as_strided((M, d_in), (ld, 1)).view(torch.float8_e4m3fn)
    far.view(torch.uint8).copy_(X.view(torch.uint8))
    compare(P.fp8_matmul(far, W, ws, x_scales=xs, y_dtype=torch.bfloat16), product(x, w), "far rows")


@pytest.mark.parametrize("yt", ["f16", "bf16"])
@pytest.mark.parametrize("M,d_out,kernel", [(5, 300, "few"), (20, 300, 32), (60, 300, 64), (130, 200, 64), (1100, 7300, 128),
                                            (2100, 8200, 256)])
def test_nan_in_16_bits(M, d_out, kernel, yt):
    """A token's NaN or infinity, a NaN code and a tile of NaN of the weights: their rows and columns, no other output's bits."""
    import torch
    from post_weight_quantization_08_amd import pipeline as P
    d_in = 1111
    assert kernel_of(M, d_in, d_out) == kernel
    dt = {"f16": torch.float16, "bf16": torch.bfloat16}[yt]
    gen = torch.Generator(device="cuda").manual_seed(M)
    W, ws, _ = codes(d_out, d_in, 128, gen)
    X = torch.randn(M, d_in, generator=gen, device="cuda")
    want = P.fp8_matmul(X, W, ws, y_dtype=dt)
    assert bool(torch.isfinite(want).all())
    X[1, 7], X[M - 2, 1110] = float("nan"), -float("inf")
    W, ws = W.clone(), ws.clone()
    W.view(torch.uint8)[d_out - 1, 1000] = 0xFF
    W.view(torch.uint8)[128:256, 512:640] = 0x7F
    ws.view(torch.uint8)[1, 4] = 255                      # as fp8_quantize leaves such a tile
    nan = torch.zeros(M, d_out, dtype=torch.bool, device="cuda")
    nan[1] = nan[M - 2] = True
    nan[:, d_out - 1] = nan[:, 128:256] = True
    got = P.fp8_matmul(X, W, ws, y_dtype=dt)
    assert torch.equal(torch.isnan(got), nan)
    assert torch.equal(got[~nan], want[~nan])
    q = P.fp8_quantize(X)
    assert torch.equal(P.fp8_matmul(q["codes"], W, ws, x_scales=q["scales"], y_dtype=dt).view(torch.int16)[~nan],
                       want.view(torch.int16)[~nan])


@pytest.mark.parametrize("M,d_out,kernel", [(4, 256, "few"), (40, 256, 64), (1100, 7300, 128), (2100, 8200, 256)])
def test_scales_far_apart_in_16_bits(M, d_out, kernel):
    """One block of the weights is 2^60 larger than all others: an output is that block's exact sum, rounded once (half a
    step, 2^-8 of it), and what the others add is below 1024 * 144 * 2^-30 = 2^-12.8."""
    import torch
    from post_weight_quantization_08_amd import pipeline as P
    nb = 9
    assert kernel_of(M, nb * 128, d_out) == kernel
    gen = torch.Generator(device="cuda").manual_seed(M)
    X, xs, x = codes(M, nb * 128, 1, gen)
    W, ws, w = codes(d_out, nb * 128, 128, gen)
    for k in range(nb):
        ws2 = ws.clone()
        s = ws2.view(torch.uint8)
        s -= 30
        s[:, k] += 60
        Y = P.fp8_matmul(X, W, ws2, x_scales=xs, y_dtype=torch.bfloat16).float()
        part = slice(k * 128, k * 128 + 128)
        want = x[:, part].double() @ w[:, part].double().t() * 2.0 ** 30
        assert bool(((Y - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -12).all()), k
