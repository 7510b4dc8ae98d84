"""The tree operators' kernels call no functions, and the register that holds
the place in LDS of a load (m0) is used nowhere but beside that load, so that
nothing of the compiler's own can be lost in it. The sources are compiled to assembly with the build's own flags."""
import os
import re
import shutil
import subprocess

import pytest

from draft_token_verification_packed_amd import build


@pytest.mark.parametrize("source", ["attention.hip", "adjust.hip", "pages.hip"])
def test_compiled_kernels(source, tmp_path):
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
    blocks = re.findall(r"ASMSTART(.*?)ASMEND", text, flags=re.S)
    loads = [b for b in blocks if "m0" in b]
    assert all(re.search(r"s_mov_b32 m0, s\d+\s+s_nop 0\s+global_load_lds_dwordx4 ", b) for b in loads)
    assert len(re.findall(r"\bm0\b", text)) == len(loads)
    assert len(re.findall("global_load_lds", text)) == len(loads)
