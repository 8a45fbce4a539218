"""fp8_matmul of few tokens on a vocabulary's outputs: tiles that fit the tokens, scales' arrays of a few bytes."""
import numpy as np
import pytest

from oracle import fp8 as F
from tests.test_gpu_fp8 import check, codes_to_torch, operands, scales_to_torch, values

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,d_in,d_out,yt", [(1, 128, 65600, "bf16"), (2, 128, 65600, "f16"), (3, 128, 65537, "f32"),
                                             (20, 256, 66000, "bf16"), (60, 128, 65600, "bf16"), (100, 256, 65600, "f32"),
                                             (130, 128, 65600, "bf16")])
def test_few_tokens_many_outputs(M, d_in, d_out, yt):
    import torch
    from post_weight_quantization_08_amd import pipeline as P
    wc, wb, w = operands(M, d_in, d_out, M)
    xc, xb = F.fp8_quantize(values(M, d_in, "f32", M, 0.7).astype(np.float64))
    dt = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[yt]
    got = P.fp8_matmul(codes_to_torch(xc), codes_to_torch(wc), scales_to_torch(wb), x_scales=scales_to_torch(xb), y_dtype=dt)
    torch.cuda.synchronize()
    check(got.double().cpu().numpy(), F.fp8_values(xc, xb), w, yt, f"{M}x{d_in}x{d_out}")
