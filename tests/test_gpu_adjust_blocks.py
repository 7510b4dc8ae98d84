"""Adjustments where a workgroup takes several rows of a request, and goes on
to its next block of them: trees and chains with penalties, biases and masks,
requests longer than all blocks side by side. Definition and tolerances as in
test_gpu_adjust.py."""
import numpy as np
import pytest

import oracle
from tests.test_gpu_adjust import _call, _case, _check
from tests.workloads import cuda_or_skip, host, to_dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def vsv():
    cuda_or_skip()
    import draft_token_verification_packed_amd as m
    m.lib()
    return m


def _both(vsv, c, **kw):
    got = _call(vsv, c, **kw)
    _check(got, c)
    x = to_dev(c["store"])
    same = _call(vsv, c, store=x, out=x, **kw)
    assert np.array_equal(host(same.float()), host(got.float()), equal_nan=True)


# (a batch's rows times slices of 2048 logits: 2 rows a block from 8192 on, or
# from 4096 on where histories are wider than 4096 tokens)
@pytest.mark.parametrize("dtype,kind,counts,V,H", [
    (oracle.F32, "wide", [3] * 200 + [64, 1], 20011, 4100),
    (oracle.BF16, "wide", [5, 1, 9, 64, 30] * 8, 14000, 4200),
    (oracle.F32, "chain", [7] * 60 + [400], 24001, 30),
    (oracle.BF16, "wide", [33] * 20, 40007, 64),
])
def test_blocks_of_several_rows(vsv, dtype, kind, counts, V, H):
    c = _case(V, counts, V, dtype, kind, 1, H=H, bias=30, tokens=300)
    print("adjust blocks %d rows V=%d H=%d dtype=%d" % (c["R"], V, H, dtype), flush=True)
    _both(vsv, c, chain=kind == "chain")
