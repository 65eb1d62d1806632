"""Registers of the 4-bit and norm kernels (no GPU needed): compiled for gfx950,
none of them may spill to memory.  Their row and tile variants are chosen so
that they do not.  (Scalar registers that go to lanes of a vector register cost
no memory and are let pass.)"""

import os
import re
import shutil
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "rotation_quantized_int8_amd", "csrc")
sys.path.insert(0, os.path.join(ROOT, "rotation_quantized_int8_amd"))


def _hipcc():
    return shutil.which("hipcc") or ("/opt/rocm/bin/hipcc" if os.path.exists("/opt/rocm/bin/hipcc") else None)


@pytest.mark.skipif(_hipcc() is None, reason="hipcc not available")
@pytest.mark.parametrize("src", ["mx_gemm.hip", "mx_rows.hip", "norm.hip"])
def test_no_kernel_spills_to_memory(src, tmp_path):
    import build   # the package's build flags
    cmd = [_hipcc(), *build.HIPCC_FLAGS, "--cuda-device-only", "-S", "-Rpass-analysis=kernel-resource-usage", "-I",
           os.path.join(ROOT, "include"), "-I", CSRC, os.path.join(CSRC, src), "-o", str(tmp_path / "out.s")]
    r = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True, timeout=600)
    assert r.returncode == 0, r.stdout[-2000:]
    name, kernels, found = None, 0, 0
    for line in r.stdout.splitlines():
        if m := re.search(r"Function Name: (\S+)", line):
            name, kernels = m.group(1), kernels + 1
        if m := re.search(r"(VGPRs Spill|ScratchSize \[bytes/lane\]): (\d+)", line):
            assert m.group(2) == "0", f"{name}: {m.group(0)}"
            found += 1
    assert kernels > 0 and found == 2 * kernels
