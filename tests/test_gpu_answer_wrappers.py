"""The wrappers of scoring, distillation and adapters: what they return and what they make of their tensors."""
import pytest

pytestmark = pytest.mark.gpu


def _allocations(f):
    import torch
    f()
    torch.cuda.synchronize()
    before = torch.cuda.memory_stats()["allocation.all.allocated"]
    f()
    return torch.cuda.memory_stats()["allocation.all.allocated"] - before


def test_a_call_allocates_each_output_and_one_workspace():
    import torch
    from post_weight_quantization_08_amd import pipeline as P
    x = torch.randn(3, 40000, device="cuda")
    assert _allocations(lambda: P.token_logprobs(x, None, 4)) <= 5 + 1
    top = P.token_logprobs(x, None, 4)
    args = (x, top["top_id"], top["top_logprob"])
    assert _allocations(lambda: P.distill_topk(*args)) <= 2 + 1
    assert _allocations(lambda: P.distill_topk(*args, want_grad=False)) <= 1 + 1


def test_without_targets_no_row_is_scored():
    """logprob is 0 for a row that is not scored, also when no row has a target, whatever the memory held before."""
    import torch
    from post_weight_quantization_08_amd import pipeline as P
    x = torch.randn(2000, 50, device="cuda")
    held = [torch.full((2000,), 3.0, device="cuda") for _ in range(8)]
    torch.cuda.synchronize()
    del held
    assert not bool(P.token_logprobs(x, None, 2)["logprob"].any())
    held = [torch.full((2000,), 3.0, device="cuda") for _ in range(8)]
    torch.cuda.synchronize()
    del held
    out, ws = P.token_logprobs_buffers(x, 2)
    assert not bool(P.token_logprobs(x, None, 2, out=out, ws=ws)["logprob"].any())
