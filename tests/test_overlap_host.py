"""Results that share memory with inputs: the test for it against a byte map,
and the refusals of tree attention. Needs no GPU."""
import os
import shutil
import subprocess

import pytest

from draft_token_verification_packed_amd import build
from tests.test_tree_host import L, _attention  # noqa: F401

HERE = os.path.dirname(os.path.abspath(__file__))


def test_strided_places_against_a_byte_map(tmp_path):
    if not shutil.which("g++"):
        pytest.skip("needs a C++ compiler")
    out = str(tmp_path / "overlap")
    subprocess.run(["g++", "-O1", "-std=c++17", "-I", build.CSRC, os.path.join(HERE, "overlap_host.cpp"), "-o", out], check=True)
    for seed in range(3):
        r = subprocess.run([out, str(seed)], capture_output=True, text=True, timeout=60)
        assert r.returncode == 0, r.stdout


# 20 rows of 8 heads of 128 bfloat16 in the first megabytes, everything else far away
FAR = dict(q=0x10000000, k=0x20000000, v=0x30000000, k_cache=0x40000000, v_cache=0x50000000, lse=0x60000000, out=0x70000000)
SPACE = dict(ws=0x80000000, wsn=1 << 30)


@pytest.mark.parametrize("bad", [
    dict(out=FAR["q"]), dict(out=FAR["q"] + 19 * 2048), dict(out=FAR["q"] - 19 * 2048), dict(out=FAR["k"]),
    dict(out=FAR["v"] + 16), dict(out=FAR["k_cache"] + 63 * 8192 + 8192 - 16), dict(out=FAR["v_cache"]), dict(out=FAR["lse"]),
    dict(out=FAR["lse"] + 20 * 8 * 4 - 16), dict(out=SPACE["ws"] + 256),
    # slices of the same rows of q, k and v that reach into one another
    dict(out=FAR["q"] + 7 * 256, q_row=4096, out_row=4096), dict(out=FAR["k"] + 256, k_row=4096, out_row=4096),
    dict(out=FAR["v"] - 7 * 256, v_row=4096, out_row=4096),
])
def test_attention_refuses_results_on_inputs(L, bad):  # noqa: F811
    assert _attention(L, **{**FAR, **SPACE, **bad}) == 1
