"""The 8-bit kernels that copy to LDS in the assembly of the built library: as
for the MXFP4 ones, only those copies may use M0; and no accumulator leaves its
registers for memory between the products."""
import os
import re

import pytest

from tests.test_mx_assembly import IMPLICIT, OBJDUMP, _kernels


@pytest.mark.skipif(not os.path.exists(OBJDUMP), reason="no llvm-objdump")
def test_only_the_copies_use_m0(tmp_path):
    kernels = _kernels(tmp_path, "fp8_")
    kernels = {s: c for s, c in kernels.items() if any("_load_lds_" in line for line in c)}
    assert sum("fp8_tile_kernel" in s for s in kernels) >= 12       # three shapes, two formats, two output types
    assert sum("fp8_few_kernel" in s for s in kernels) >= 20        # ten shapes, two formats
    for symbol, code in kernels.items():
        copies = 0
        for i, line in enumerate(code):
            if line.startswith("global_load_lds_dwordx4 "):
                assert code[i - 1] == "s_nop 0" and re.fullmatch(r"s_mov_b32 m0, s\d+", code[i - 2]), symbol
                copies += 1
            else:
                assert not IMPLICIT.search(line), (symbol, line)
        assert copies > 0 and sum("m0" in line for line in code) == copies, symbol
        # the main loop: from the first product to the last, no scratch access
        products = [i for i, line in enumerate(code) if line.startswith("v_mfma_scale_f32_")]
        assert not any("scratch" in line for line in code[products[0]:products[-1]]), symbol
