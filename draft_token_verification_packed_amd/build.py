"""Build the HIP library `libvspec_verify.so` in-tree for gfx950.

Run `python -m draft_token_verification_packed_amd.build` (or call build())
on any machine with ROCm's hipcc; no GPU is needed to compile.
"""
import os
import shutil
import subprocess
import sys
import tempfile

PKG = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(os.path.dirname(PKG), "include")
LIB = os.path.join(PKG, "libvspec_verify.so")
SOURCES = ["abi.cpp", "verify.hip", "sampled.hip", "probabilistic.hip", "confidence.hip", "draw.hip", "top.hip", "distill.hip",
           "allocate.hip", "goodput.cpp", "static_ws.hip"]
ARCH = "gfx950"
# Packed-FP32 VALU forms are kept out of the code objects: the compiler would
# otherwise fuse float pairs into v_pk_* instructions.
FLAGS = ["-O3", "-std=c++17", "-fPIC", "--offload-arch=" + ARCH,
         "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
         "-Wall", "-Wno-unused-function"]
# The queue kernels loop over rows: with loop-invariant code motion the
# compiler hoists a hundred constants out of that loop into registers, and
# the sampled kernel no longer fits two workgroups per CU while the
# probabilistic one spills 23 VGPRs (48 instead of 144 bytes of scratch per
# lane without it; 581 instead of 609 us on the mixed B=512, K=7 batch).
# The draws' kernels hold several searches one after another, whose constants
# are hoisted to the kernel's start the same way: 18 to 60 VGPRs spill with it
# and none without (512 bf16 rows with top-p 58 instead of 61.5 us, 128 fp32
# rows with every filter 53 instead of 56).
_NO_LICM = ["-mllvm", "-disable-machine-licm"]
SOURCE_FLAGS = {"sampled.hip": _NO_LICM, "probabilistic.hip": _NO_LICM, "draw.hip": _NO_LICM}


def hipcc():
    p = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
    if not os.path.exists(p):
        raise RuntimeError("hipcc not found: ROCm is required to build the library")
    return p


def _run(cmd):
    r = subprocess.run(cmd, capture_output=True, text=True)
    noise = "is not a recognized feature for this target"
    msgs = "\n".join(l for l in (r.stdout + r.stderr).splitlines() if noise not in l)
    if r.returncode != 0:
        raise RuntimeError("hipcc failed:\n" + msgs)
    return msgs


def build(extra_flags=(), out=LIB, verbose=False):
    """Compile every source to an object (with its own flags) and link the library."""
    objdir = tempfile.mkdtemp(prefix="vsv_build_")
    try:
        objs, msgs = [], []
        for s in SOURCES:
            obj = os.path.join(objdir, s + ".o")
            cmd = ([hipcc()] + FLAGS + SOURCE_FLAGS.get(s, []) + list(extra_flags) +
                   ["-I", CSRC, "-I", INCLUDE, "-c", os.path.join(CSRC, s), "-o", obj])
            msgs.append(_run(cmd))
            objs.append(obj)
        msgs.append(_run([hipcc(), "-shared", "-fPIC", "--offload-arch=" + ARCH] + objs + ["-o", out + ".tmp"]))
    finally:
        shutil.rmtree(objdir, ignore_errors=True)
    if verbose and any(m.strip() for m in msgs):
        print("\n".join(m for m in msgs if m.strip()), file=sys.stderr)
    os.replace(out + ".tmp", out)
    return out


if __name__ == "__main__":
    print(build(verbose=True))
