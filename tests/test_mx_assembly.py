"""The MXFP4 tile kernels in the assembly of the built library.

Their copies to LDS set M0 in inline assembly, which cannot name it as
clobbered, so nothing that the compiler generates there may use it."""
import os
import re
import shutil
import subprocess

import pytest

from bit_companded_adam_amd import flashopt as F

OBJDUMP = os.path.join(os.environ.get("ROCM_PATH", "/opt/rocm"), "llvm", "bin", "llvm-objdump")
# instructions of a kernel that read M0 without naming it
IMPLICIT = re.compile(r"movrel|s_set_gpr_idx|ds_gws|ds_append|ds_consume|ds_ordered|addtid|s_sendmsg|v_interp|"
                      r"buffer_load\S* .*\blds\b|_load_lds_")


def _kernels(tmp_path, name):
    """{symbol: instructions} of the device functions whose symbol holds name."""
    if not os.path.exists(F._LIB_PATH):
        import __graft_entry__
        __graft_entry__.build()
    lib = shutil.copy(F._LIB_PATH, tmp_path)
    subprocess.run([OBJDUMP, "--offloading", lib], check=True, capture_output=True, cwd=tmp_path)
    found, code = {}, None
    for part in sorted(tmp_path.glob("*gfx950*")):
        text = subprocess.run([OBJDUMP, "-d", "--no-show-raw-insn", str(part)], check=True, capture_output=True,
                              text=True).stdout
        for line in text.splitlines():
            head = re.match(r"[0-9a-f]+ <(\S+)>:", line)
            if head:
                code = found.setdefault(head.group(1), []) if name in head.group(1) else None
            elif code is not None and line.startswith("\t"):
                code.append(line.split("//")[0].strip())
    return found


@pytest.mark.skipif(not os.path.exists(OBJDUMP), reason="no llvm-objdump")
def test_only_the_copies_use_m0(tmp_path):
    kernels = _kernels(tmp_path, "mx_tile_kernel")
    assert len(kernels) >= 8                     # four tile shapes, two output types
    for symbol, code in kernels.items():
        copies = 0
        for i, line in enumerate(code):
            if line.startswith("global_load_lds_dwordx4 "):
                assert code[i - 1] == "s_nop 0" and re.fullmatch(r"s_mov_b32 m0, s\d+", code[i - 2]), symbol
                copies += 1
            else:
                assert not IMPLICIT.search(line), (symbol, line)
        assert copies > 0 and sum("m0" in line for line in code) == copies, symbol
