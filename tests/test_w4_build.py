"""The built kernels of the products with 4-bit weights keep their values in
registers (CPU only: from the metadata of the code objects in the library)."""

import os
import re
import subprocess

import pytest

import mixture_experts_ffn_moe_amd as moe

READELF = "/opt/rocm/llvm/bin/llvm-readelf"
EM_AMDGPU = 224


def scratch_bytes(tmp_path):
    """Scratch memory of each kernel in the library, bytes a lane."""
    with open(moe.LIB_PATH, "rb") as f:
        lib = f.read()
    sizes = {}
    for m in re.finditer(b"\x7fELF", lib):
        at = m.start()
        if int.from_bytes(lib[at + 18:at + 20], "little") != EM_AMDGPU:
            continue
        obj = tmp_path / "object"
        obj.write_bytes(lib[at:])
        notes = subprocess.run([READELF, "--notes", str(obj)], capture_output=True, text=True).stdout
        for name, size in re.findall(r"\.name:\s+(\S+)\s+\.private_segment_fixed_size:\s+(\d+)", notes):
            sizes[name] = int(size)
    return sizes


@pytest.mark.skipif(not os.path.exists(READELF), reason="needs llvm-readelf")
def test_no_scratch(tmp_path):
    sizes = {n: b for n, b in scratch_bytes(tmp_path).items() if "k_w4" in n}
    assert len(sizes) > 90
    assert not {n: b for n, b in sizes.items() if b}
