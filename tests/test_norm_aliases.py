"""What the norm's kernels promise the compiler about their pointers: nothing
that a call may break.  dx may be dy or dh itself, and h may be x or residual;
only the workspace of the backward pass and dgain are apart from all else."""
import os
import re
import subprocess

import pytest

from bit_companded_adam_amd import _build

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")


@pytest.mark.skipif(not os.path.exists(HIPCC), reason="no hipcc")
def test_only_what_is_apart_is_restrict(tmp_path):
    flags = [f for f in _build.HIPCC_FLAGS if f not in ("-shared", "-Wall", "-O3")]
    out = tmp_path / "norm.ll"
    subprocess.check_call([HIPCC, *flags, "-O0", "-S", "-emit-llvm", "--cuda-device-only", "-I",
                           os.path.join(_build.ROOT, "include"), "-I", _build.CSRC,
                           os.path.join(_build.CSRC, "flashopt_norm.hip"), "-o", str(out)],
                          stderr=subprocess.DEVNULL)
    heads = [line for line in out.read_text().splitlines() if line.startswith("define") and "amdgpu_kernel" in line]
    seen = {}
    for line in heads:
        kernel = re.search(r"rms_norm_backward_kernel|rms_norm_kernel|norm_gain_kernel", line)
        if kernel:
            seen.setdefault(kernel.group(), set()).add(tuple(map(int, re.findall(r"noalias [^%]*%(\d+)", line))))
    # by number: the backward pass's arguments are its inputs, dx, dx's stride
    # and the workspace; norm_gain_kernel's the workspace, ..., dgain
    assert seen == {"rms_norm_kernel": {()}, "rms_norm_backward_kernel": {(3,)}, "norm_gain_kernel": {(0, 3)}}
