"""Sizes of the adapters' gradients that one launch could not hold are refused before anything is enqueued."""
import pytest

from tests.test_abi_cpu import G  # noqa: F401  (fixture)
from tests.test_abi_lora_grad_cpu import _lg


def test_many_adapters_on_wide_layers(G):
    half = 1 << 18
    assert _lg(G, n=1024, d_in=half, d_out=half + 1, r=1) == G.EUNSUPPORTED
    assert _lg(G, n=1024, d_in=half, d_out=half, r=1, ws_bytes=0) == G.ENOMEM      # the last that is served
    with pytest.raises(G.GptqError):
        G.gptq_lora_grad_workspace_size(4, half, half + 1, 1, 1024)
    assert G.gptq_lora_grad_workspace_size(4, half, half, 1, 1024) > 0
    assert G.gptq_lora_grad_workspace_size(4, 1 << 22, 1 << 22, 1, 64) > 0
