"""Every tile shape of the 8-bit product is in the built library, in both formats
of the first operand (and both output types), and no other: a shape that no rule
reaches is none to keep."""
import os
import re

import pytest

from tests.test_mx_assembly import OBJDUMP, _kernels


@pytest.mark.skipif(not os.path.exists(OBJDUMP), reason="no llvm-objdump")
def test_shapes(tmp_path):
    seen = {"fp8_tile_kernel": set(), "fp8_few_kernel": set()}
    for symbol in _kernels(tmp_path, "fp8_"):
        named = re.search(r"(fp8_tile_kernel|fp8_few_kernel)I(\w+?)EEv", symbol)
        if named:
            seen[named.group(1)].add(tuple(int(n) for n in re.findall(r"L[bi](\d+)", named.group(2))))
    # output type and format; rows of B, rows of A, wavefronts along each
    tiles = [(256, 256, 4, 2), (256, 192, 4, 2), (128, 128, 2, 2), (64, 64, 2, 2)]
    assert seen["fp8_tile_kernel"] == {(f32, kind, *t) for t in tiles for f32 in (0, 1) for kind in (0, 1)}
    # tiles of 16 rows: of A, of B
    few = [(1, 1), (2, 1), (1, 2), (2, 2), (1, 4), (3, 2), (2, 4), (4, 2), (3, 4), (4, 4)]
    assert seen["fp8_few_kernel"] == {(kind, *t) for t in few for kind in (0, 1)}
