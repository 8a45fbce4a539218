"""Registers and LDS of the 8-bit operators, the policy loss and the adapters' gradients, as built: no register of theirs is
spilled, but for a few before and behind the loops of the kernels that fill the register file."""
import pytest

from tests.test_kernel_resources import _kernels

NAMES = ("fp8_rows_kernel", "fp8_tiles_kernel", "fp8_few_kernel", "fp8_tile_kernel", "fp8_big_kernel", "fp8_join_kernel",
         "policy_row_kernel", "policy_part_kernel", "lora_grad_project_kernel", "lora_grad_terms_kernel",
         "lora_grad_outer_kernel", "lora_grad_join_kernel", "lora_grad_input_kernel")


# 256 tokens by 256 rows; the sums over tokens of 64 ranks with 16-bit rows
FULL = {"fp8_big_kernel": ("", 6), "fp8_tile_kernel": ("Li256ELi256E", 2), "lora_grad_outer_kernel": ("ILi", 3)}


@pytest.mark.parametrize("name", NAMES)
def test_spills_and_lds(name):
    found = {k: v for k, v in _kernels().items() if name in k}
    assert found, name
    for k, v in found.items():
        which, most = FULL.get(name, ("", 0))
        allowed = most if which in k else 0
        assert v[".vgpr_spill_count"] <= allowed, (k, v[".vgpr_spill_count"])
        assert v[".group_segment_fixed_size"] <= 160 * 1024, k
