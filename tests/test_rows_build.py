"""The row operators' kernels are compiled as one function each.

In a called device function of more than 128 KB the compiler's long branches
use the registers that hold the return address, so the function returns into
nowhere; a kernel that calls nothing cannot get there. The sources are
compiled to assembly with the build's own flags and searched for calls."""
import os
import shutil
import subprocess

import pytest

from draft_token_verification_packed_amd import build


@pytest.mark.parametrize("source", ["draw.hip", "top.hip", "distill.hip"])
def test_kernels_call_no_functions(source, tmp_path):
    if not (shutil.which("hipcc") or os.path.exists("/opt/rocm/bin/hipcc")):
        pytest.skip("needs hipcc")
    out = tmp_path / "device.s"
    cmd = ([build.hipcc()] + build.FLAGS + build.SOURCE_FLAGS.get(source, []) +
           ["-I", build.CSRC, "-I", build.INCLUDE, "-S", "--cuda-device-only", os.path.join(build.CSRC, source), "-o",
            str(out)])
    subprocess.run(cmd, check=True, stdout=subprocess.DEVNULL, stderr=subprocess.DEVNULL)
    text = out.read_text()
    assert ".amdhsa_kernel" in text
    assert "s_swappc" not in text
