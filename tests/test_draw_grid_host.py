"""The borders of the draw's bins, in a host build of the kernel's own header:
at every temperature that is accepted the search for a border ends, at the
least float of the bin. Where a bin is narrower than the smallest float, the
search starts at zero, and has to step past both zeros."""
import os
import shutil
import subprocess

import pytest

from draft_token_verification_packed_amd import build

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    if not (shutil.which("hipcc") or os.path.exists("/opt/rocm/bin/hipcc")):
        pytest.skip("needs hipcc")
    out = str(tmp_path_factory.mktemp("grid") / "draw_grid")
    subprocess.run([build.hipcc(), "-O2", "-std=c++17", "-I", build.CSRC, "--offload-arch=" + build.ARCH,
                    os.path.join(HERE, "draw_grid_host.cpp"), "-o", out], check=True)
    return out


@pytest.mark.parametrize("T", ["1.4e-45", "1e-44", "8e-44", "9e-44", "1e-43", "1e-42", "1e-40", "1.2e-38", "1e-30", "0.05", "1",
                               "1000", "3e38"])
def test_borders_are_found_at_every_temperature(program, T):
    r = subprocess.run([program, T], capture_output=True, text=True, timeout=20)
    assert r.returncode == 0, r.stdout
