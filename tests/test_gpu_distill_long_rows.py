"""Distillation of rows too long for a workgroup's registers alone, several rows
to a workgroup: unusual rows next to ordinary ones."""
import numpy as np
import pytest

import oracle as O
from tests import answer_data as D
from tests.gpu_run import log

pytestmark = pytest.mark.gpu


# vocabularies on both sides of 16 and of 20 blocks of 16 bytes per thread
@pytest.mark.parametrize("want_grad", [True, False])
@pytest.mark.parametrize("V,dtype", [(131072, "bf16"), (131080, "f16"), (151936, "bf16"), (163840, "f16"), (163848, "bf16"),
                                     (65541, "f32"), (81920, "f32"), (81923, "f32")])
def test_unusual_rows_next_to_ordinary_ones(V, dtype, want_grad):
    import torch
    from post_weight_quantization_08_amd import pipeline as P
    k, n = 40, 600
    kinds = ["plain", "lowest_but_one", "peaked", "plain", "masked", "plain", "large", "plain", "far"]
    xs = D.rows(kinds, V, dtype, 51)
    x = D.exact(xs, dtype)
    ids, lps = D.teacher(x, k, 1.0, 51, True)
    x[3, V - 3] = np.nan
    x[5] = -np.inf
    weight = np.ones(len(kinds), dtype=np.float32)
    weight[7] = 0.0
    xs = D.store(x, dtype)
    o = O.distill_topk(x, ids, lps, 1.0, True, weight)
    loss_b, grad_b = D.distill_bounds(x, ids, lps, 1.0, True, weight, o, dtype)
    take = torch.arange(n, device="cuda") % len(kinds)
    out = P.distill_topk(D.to_torch(xs, dtype)[take], torch.from_numpy(ids).cuda()[take], torch.from_numpy(lps).cuda()[take],
                         weight=torch.from_numpy(weight).cuda()[take], want_grad=want_grad)
    torch.cuda.synchronize()
    for name, b in (("loss", loss_b), ("grad", grad_b)):
        if name not in out:
            continue
        got, want = out[name][:len(kinds)].double().cpu().numpy(), o[name]
        np.testing.assert_array_equal(np.isnan(got), np.isnan(want))
        fine = np.isfinite(want)
        np.testing.assert_array_equal(got[~fine & ~np.isnan(want)], want[~fine & ~np.isnan(want)])
        worst = float((np.abs(got[fine] - want[fine]) / np.maximum(b[fine], 1e-300)).max())
        log(f"[gpu] distill long rows {V} {dtype} {name}: worst error / bound {worst:.3f}")
        assert worst <= 1
        # a row that starts alike sums in the same order: rows 8 apart, and the kinds repeat every nine
        bits = out[name].view(torch.int32 if out[name].dtype == torch.float32 else torch.int16)
        assert torch.equal(bits, bits[torch.arange(n, device="cuda") % (8 * len(kinds))])
