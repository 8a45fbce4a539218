"""What the compiler made of the kernels whose speed rests on registers, from the metadata of the built library."""
import glob
import os
import struct

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "post_weight_quantization_08_amd", "libgptq.so")
EM_AMDGPU = 224
NT_AMDGPU_METADATA = 32


def _unpack(b, at=0):
    """One MessagePack value (the forms the metadata uses) and where it ends."""
    t = b[at]
    at += 1
    if t < 0x80:
        return t, at
    if t >= 0xE0:
        return t - 0x100, at
    if t in (0xC0, 0xC2, 0xC3):
        return {0xC0: None, 0xC2: False, 0xC3: True}[t], at
    ints = {0xCC: ">B", 0xCD: ">H", 0xCE: ">I", 0xCF: ">Q", 0xD0: ">b", 0xD1: ">h", 0xD2: ">i", 0xD3: ">q"}
    if t in ints:
        return struct.unpack_from(ints[t], b, at)[0], at + struct.calcsize(ints[t])
    for first, last, wide, kind in ((0xA0, 0xBF, {0xD9: ">B", 0xDA: ">H", 0xDB: ">I"}, "text"),
                                    (0x90, 0x9F, {0xDC: ">H", 0xDD: ">I"}, "list"),
                                    (0x80, 0x8F, {0xDE: ">H", 0xDF: ">I"}, "map")):
        if first <= t <= last:
            n = t - first
        elif t in wide:
            n = struct.unpack_from(wide[t], b, at)[0]
            at += struct.calcsize(wide[t])
        else:
            continue
        if kind == "text":
            return b[at:at + n].decode(), at + n
        out = []
        for _ in range(n * (2 if kind == "map" else 1)):
            v, at = _unpack(b, at)
            out.append(v)
        return (dict(zip(out[::2], out[1::2])) if kind == "map" else out), at
    raise ValueError(hex(t))


def _kernels():
    """{kernel name: its metadata} of every gfx950 code object in the library."""
    b = open(LIB, "rb").read()
    found, at = {}, b.find(b"\x7fELF", 1)
    while at >= 0:
        if struct.unpack_from("<H", b, at + 18)[0] == EM_AMDGPU:
            phoff, = struct.unpack_from("<Q", b, at + 32)
            size, count = struct.unpack_from("<HH", b, at + 54)
            for i in range(count):
                kind, _, off, _, _, length = struct.unpack_from("<IIQQQQ", b, at + phoff + i * size)
                if kind != 4:                                    # PT_NOTE
                    continue
                p, end = at + off, at + off + length
                while p < end:
                    n_name, n_desc, note = struct.unpack_from("<III", b, p)
                    desc = p + 12 + (n_name + 3) // 4 * 4
                    if note == NT_AMDGPU_METADATA and b[p + 12:p + 18] == b"AMDGPU":
                        for k in _unpack(b[desc:desc + n_desc])[0]["amdhsa.kernels"]:
                            found[k[".name"]] = k
                    p = desc + (n_desc + 3) // 4 * 4
        at = b.find(b"\x7fELF", at + 1)
    return found


@pytest.fixture(scope="module")
def kernels():
    if not os.path.exists(LIB):
        pytest.skip("the library is not built")
    assert glob.glob(os.path.join(ROOT, "post_weight_quantization_08_amd", "csrc", "*.hip"))
    k = _kernels()
    assert len(k) > 100
    return k


def test_rows_of_distillation_stay_in_registers(kernels):
    """A lane's block is four registers: no kernel that holds a row spills one (up to three scalars once a row)."""
    rows = {n: k for n, k in kernels.items() if "distill_row_kernel" in n}
    assert len(rows) == 3 * 5 * 2
    spilled = {n: k[".vgpr_spill_count"] for n, k in rows.items() if k[".vgpr_spill_count"] >= 4}
    assert not spilled, spilled


@pytest.mark.parametrize("name", ["logprobs_kernel", "logprobs_join_kernel", "distill_part_kernel", "lora_down_kernel",
                                  "lora_down_lds_kernel", "lora_up_kernel", "lora_up_few_kernel", "lora_down_few_kernel",
                                  "w4_main_kernel", "w4_wide_kernel", "w4_stage_kernel"])
def test_kernels_without_spills(kernels, name):
    mine = {n: k for n, k in kernels.items() if name in n}
    assert mine
    assert not {n: k[".vgpr_spill_count"] for n, k in mine.items() if k[".vgpr_spill_count"]}
