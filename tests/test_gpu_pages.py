"""Block tables and slots against the oracle; every output is exact."""
import numpy as np
import pytest

import oracle
from tests.workloads import cuda_or_skip, host, to_dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def vsv():
    cuda_or_skip()
    import draft_token_verification_packed_amd as m
    m.lib()
    return m


def _state(rng, B, page, most, rows_hi, spare):
    length = rng.integers(0, most + 1, B).astype(np.int32)
    rows = rng.integers(0, rows_hi + 1, B)
    held = -(-length // page) + rng.choice([0, 0, 0, 1, 3], B)
    gone = rng.random(B) < 0.2
    length[gone], rows[gone] = 0, 0
    W = int(held.max(initial=0)) + rows_hi // page + 3
    pool = int(held.sum()) + spare
    ids = rng.permutation(pool).astype(np.int32)
    table = np.full((B, W), -1, dtype=np.int32)
    at = 0
    for i in range(B):
        table[i, :held[i]] = ids[at:at + held[i]]
        at += held[i]
    free = np.full(max(pool, 1), -1, dtype=np.int32)
    free[:pool - at] = ids[at:]
    off = np.concatenate(([0], np.cumsum(rows))).astype(np.int32)
    return table, held.astype(np.int32), length, off, free, np.array([pool - at], dtype=np.int32), page


def _check(vsv, state, num_rows):
    table, held, length, off, free, count, page = state
    ref = oracle.plan_pages(table, held, length, off, free, count[0], page, num_rows)
    d = [to_dev(a) for a in state[:-1]]
    for again in range(2):            # repeated on the same inputs: the same results
        out = vsv.plan_pages(*d, page, num_rows)
        for k in ("slot", "position", "held", "length", "free_count"):
            assert np.array_equal(host(out[k]), ref[k]), (k, again)
        assert np.array_equal(host(d[0]), ref["block_table"])
        assert np.array_equal(host(d[4]), ref["free_pages"])
        assert int(host(out["error_flag"])[0]) == (vsv.FLAG_PAGES if ref["short"] else 0)
    return ref


@pytest.mark.parametrize("B,page,most,rows_hi,spare", [
    (1, 16, 0, 0, 0), (1, 1, 5, 3, 9), (4, 16, 100, 5, 20), (130, 16, 500, 8, 400), (256, 64, 4000, 300, 2000),
    (257, 7, 300, 9, 2000), (1500, 32, 200, 3, 1600), (8192, 16, 40, 2, 9000), (3, 128, 9, 9000, 300),
])
def test_plans_match_the_oracle(vsv, B, page, most, rows_hi, spare):
    rng = np.random.default_rng(B + page)
    state = _state(rng, B, page, most, rows_hi, spare)
    print("pages B=%d page=%d rows=%d" % (B, page, state[3][-1]), flush=True)
    _check(vsv, state, int(state[3][-1]) + 5)


@pytest.mark.parametrize("B,spare", [(6, 0), (40, 3), (300, 40)])
def test_a_pool_that_runs_out(vsv, B, spare):
    state = _state(np.random.default_rng(spare), B, 4, 30, 30, spare)
    assert _check(vsv, state, int(state[3][-1]))["short"]


def test_steps_in_a_row(vsv):
    """A serving loop: the state behind a call is the next call's."""
    rng = np.random.default_rng(7)
    B, W, page, pool = 24, 12, 8, 200
    table = to_dev(np.full((B, W), -1, dtype=np.int32))
    free = to_dev(rng.permutation(pool).astype(np.int32))
    held, length = [to_dev(np.zeros(B, dtype=np.int32)) for _ in range(2)]
    count = to_dev(np.array([pool], dtype=np.int32))
    for step in range(12):
        state = [host(t).copy() for t in (table, held, length)]
        rows = rng.integers(0, 7, B)
        over = rng.random(B) < 0.15
        state[2][over] = 0
        length = to_dev(state[2])
        rows[over] = 0
        off = np.concatenate(([0], np.cumsum(rows))).astype(np.int32)
        ref = oracle.plan_pages(*state, off, host(free), host(count)[0], page, 170)
        out = vsv.plan_pages(table, held, length, to_dev(off), free, count, page, 170)
        for k in ("slot", "position", "held", "length", "free_count"):
            assert np.array_equal(host(out[k]), ref[k]), (k, step)
        held, length, count = out["held"], out["length"], out["free_count"]


def test_device_conditions(vsv):
    def flag(**kw):
        rng = np.random.default_rng(3)
        names = ("table", "held", "length", "off", "free", "count")
        s = dict(zip(names, _state(rng, 5, 4, 30, 6, 40)))
        s["length"][:] = 10
        s["held"][:] = 3
        s["off"] = np.array([0, 2, 4, 6, 8, 10], dtype=np.int32)
        s["table"] = np.arange(5 * 8, dtype=np.int32).reshape(5, 8)
        s.update(kw)
        out = vsv.plan_pages(*[to_dev(s[n]) for n in names], 4, 10)
        return int(host(out["error_flag"])[0]), {k: host(v) for k, v in out.items()}
    i32 = lambda *a: np.array(a, dtype=np.int32)
    assert flag()[0] == 0
    for bad in (dict(off=i32(0, 2, 1, 6, 8, 10)), dict(off=i32(0, 2, 4, 6, 8, 11)), dict(length=i32(10, -1, 10, 10, 10)),
                dict(held=i32(3, 9, 3, 3, 3)), dict(length=i32(31, 10, 10, 10, 10)), dict(count=i32(-1)),
                dict(length=i32(2 ** 31 - 1, 10, 10, 10, 10)), dict(table=np.full((5, 8), -1, dtype=np.int32)),
                dict(count=i32(10 ** 6))):
        bits, out = flag(**bad)
        assert bits & vsv.FLAG_LAYOUT, bad
    bits, out = flag(length=i32(31, 10, 10, 10, 10))
    assert out["length"].tolist() == [31, 12, 12, 12, 12] and out["slot"][:2].tolist() == [-1, -1]


def test_no_requests(vsv):
    import torch
    z = torch.zeros(0, dtype=torch.int32, device="cuda")
    count = to_dev(np.array([3], dtype=np.int32))
    out = vsv.plan_pages(torch.zeros((0, 4), dtype=torch.int32, device="cuda"), z, z, to_dev(np.zeros(1, dtype=np.int32)),
                         to_dev(np.arange(5, dtype=np.int32)), count, 16, 3)
    assert host(out["slot"]).tolist() == [-1] * 3 and host(out["free_count"]).tolist() == [3]
