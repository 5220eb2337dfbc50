"""The built kernels of the general router, of the 8-bit quantizers and of the
8-bit linear layers keep their values in registers (CPU only)."""

import os

import pytest

from tests.test_w4_build import READELF, scratch_bytes

# kernels, and at least how many forms of each the types and options make
FORMS = {"k_route_topkI": 72, "k_route_topk_backward": 15, "k_quant_rows": 12, "k_quant_tile": 24,
         "k_fp8_rows": 24, "k_fp8_stay": 16, "k_fp8_tile": 64}


@pytest.mark.skipif(not os.path.exists(READELF), reason="needs llvm-readelf")
def test_no_scratch(tmp_path):
    sizes = scratch_bytes(tmp_path)
    for name, forms in FORMS.items():
        of = {n: b for n, b in sizes.items() if name in n}
        assert len(of) >= forms, (name, len(of))
        assert not {n: b for n, b in of.items() if b}
