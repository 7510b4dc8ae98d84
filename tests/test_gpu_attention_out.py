"""Where tree attention may put its results: beside its inputs in the same
rows or heads, but on none of them."""
import pytest

import oracle
from tests.test_gpu_attention import _call, _case, _check
from tests.workloads import cuda_or_skip, to_dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def vsv():
    cuda_or_skip()
    import draft_token_verification_packed_amd as m
    m.lib()
    return m


@pytest.mark.parametrize("dtype", [oracle.F32, oracle.BF16])
@pytest.mark.parametrize("heads_first", [False, True])
def test_results_beside_the_inputs(vsv, dtype, heads_first):
    import torch
    c = _case(60, [7, 30, 12], [90, 0, 33], 6, 2, 64, 16, dtype)
    q, k, v = [to_dev(c[n]) for n in ("q", "k", "v")]
    # [rows, heads of q, k, v and out between one another, dim]
    wide = torch.zeros((16, 49, 64) if heads_first else (49, 16, 64), dtype=q.dtype, device="cuda")
    rows = wide.transpose(0, 1) if heads_first else wide
    at = dict(q=rows[:, 0:12:2], out=rows[:, 1:12:2], k=rows[:, 12:14], v=rows[:, 14:16])
    for n, t in (("q", q), ("k", k), ("v", v)):
        at[n].copy_(t)
    got, lse = _call(vsv, c, **at)
    assert got.data_ptr() == at["out"].data_ptr()
    _check(got, lse, c)
    for n, t in (("q", q), ("k", k), ("v", v)):
        assert torch.equal(at[n], t)
    for n in ("q", "k", "v"):
        bad = at[n] if n == "q" else rows[:, 9:15] if n == "k" else rows[:, 10:16]
        with pytest.raises(vsv.VSVError):
            _call(vsv, c, **dict(at, out=bad))
    kc = to_dev(c["kc"])
    with pytest.raises(vsv.VSVError):
        _call(vsv, c, **dict(at, kc=kc, out=kc.view(-1)[:49 * 6 * 64].view(49, 6, 64)))
