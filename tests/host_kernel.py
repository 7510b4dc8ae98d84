"""Builds of a kernel's own source for the CPU (hip_on_host/): launches and the
statements in assembly become calls of the stand-in, all else is compiled as it
stands."""
import os
import re
import shutil
import subprocess

import pytest

from draft_token_verification_packed_amd import build

HERE = os.path.dirname(os.path.abspath(__file__))
# assembly statements and what stands in for them
ASM = ((r'"s_mov_b32 m0, %0\\n\\t".*?;', "emu::load_to_lds(from, to);"),
       (r'"s_waitcnt vmcnt\(%0\) lgkmcnt\(0\)".*?;', "emu::wait_loads(N);"),
       (r'"s_waitcnt lgkmcnt\(0\)".*?;', "emu::meet();"))


def compiler():
    p = os.path.join(os.path.dirname(os.path.realpath(shutil.which("hipcc") or "/opt/rocm/bin/hipcc")), "..", "llvm", "bin",
                     "clang++")
    if not os.path.exists(p):
        pytest.skip("needs ROCm's compiler")
    return p


def program(tmp, source, main, edits=()):
    """Compiles tests/`main`, which includes kernel.hpp: the text of
    csrc/`source` with `edits` (pairs of texts) made first."""
    text = open(os.path.join(build.CSRC, source)).read()
    for old, new in edits:
        assert old in text, old
        text = text.replace(old, new)
    for pattern, call in ASM:
        text = re.sub(r"asm volatile\(\s*" + pattern, call, text, flags=re.S)
    assert "asm" not in re.sub(r"//.*", "", text)
    text, launches = re.subn(r"(\w+<[^<>;]*>)\s*<<<(.*?), 0, s>>>\(a\);", r"emu::launch(\1, \2, a);", text, flags=re.S)
    assert launches and "<<<" not in text
    open(os.path.join(str(tmp), "kernel.hpp"), "w").write(text)
    out = os.path.join(str(tmp), main + ".out")
    # (addresses in LDS are 32 bits, so the program lies below 2^31; whole numbers wrap as the device's do)
    subprocess.run([compiler(), "-O2", "-std=c++17", "-fwrapv", "-fno-pie", "-no-pie", "-w", "-I", os.path.join(HERE, "hip_on_host"),
                    "-I", str(tmp), "-I", build.CSRC, "-I", build.INCLUDE, os.path.join(HERE, main), "-o", out], check=True)
    return out


def run(program, *args, timeout=300):
    r = subprocess.run([program] + [str(a) for a in args], capture_output=True, text=True, timeout=timeout)
    assert r.returncode == 0, "%d\n%s%s" % (r.returncode, r.stdout[-2000:], r.stderr[-2000:])
    return r.stdout
