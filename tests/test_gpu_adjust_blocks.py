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


@pytest.mark.parametrize("kind", ["chain", "wide"])
@pytest.mark.parametrize("counts,empty", [([5, 4, 3], 2), ([2], 3), ([1, 1, 6], 9)])
def test_requests_without_rows_leave_every_draft(vsv, kind, counts, empty):
    """No padding rows: the batch ends with the last request that has rows,
    and holds more drafts than rows less requests."""
    import torch
    c = _case(21, counts, 300, oracle.F32, kind, tokens=40)
    c["off"] = np.concatenate((c["off"], np.full(empty, c["off"][-1], dtype=np.int32)))
    for k in ("history", "history_len", "prompt_len", "repetition", "frequency", "presence"):
        c[k] = np.concatenate((c[k], np.repeat(c[k][:1], empty, 0)))
    c["bias_offsets"] = np.concatenate((c["bias_offsets"], np.repeat(c["bias_offsets"][-1:], empty)))
    assert len(c["drafts"]) == c["R"] - len(counts) > c["R"] - len(counts) - empty
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    _check(_call(vsv, c, chain=kind == "chain", error_flag=err), c)
    assert int(err) == 0
    for n in (c["R"] + 1, c["R"] - len(counts) - empty - 1):
        if c["R"] > len(counts) + empty and n >= 0:
            with pytest.raises(ValueError):
                _call(vsv, dict(c, drafts=np.zeros(n, dtype=np.int32)))


def test_drafts_of_single_rows_are_not_read(vsv):
    c = _case(22, [1] * 5, 300, oracle.F32)
    want = host(_call(vsv, c))
    for n in (0, 3, 9):
        assert np.array_equal(host(_call(vsv, dict(c, drafts=np.full(n, 7, dtype=np.int32)))), want, equal_nan=True)
