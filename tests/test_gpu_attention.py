"""Attention of draft trees over a paged cache against the float64 definition.

Tolerances. A score is a sum of D products, each factor exact, in float32: it
is off by at most D 2^-24 sum |q k| (any order of adding), E in all once
scaled and rounded, and exp2 and its argument add 2^-22 (1 + |s|). Weights
are then off by a factor of 1 + e, e = 2 E + 2^-21 (1 + max |s|), so is their sum; bfloat16
weights are rounded (half a step, 2^-8, is asked of each), and sums over T tokens add
T 2^-24. The output is a mean of values with those weights:
  |out - exact| <= (2 e + h + T 2^-23) sum p |v| + half a step of the value,
h = 2^-8 for bfloat16 and 0 for float32; lse is off by at most
e + 2^-22 (1 + |lse|)."""
import numpy as np
import pytest

import oracle
import synth
from tests.tree_cases import layout
from tests.workloads import cuda_or_skip, host, to_dev

pytestmark = pytest.mark.gpu

F32, BF16 = oracle.F32, oracle.BF16


@pytest.fixture(scope="module")
def vsv():
    cuda_or_skip()
    import draft_token_verification_packed_amd as m
    m.lib()
    return m


def _bits(x, dtype):
    x = np.ascontiguousarray(x, dtype=np.float32)
    return synth.f32_to_bf16_bits(x.reshape(1, -1)).reshape(x.shape) if dtype == BF16 else x


def _case(seed, counts, lens, H, KV, D, page, dtype, kind="wide", spread=1.0):
    rng = np.random.default_rng(seed)
    off, owner, par = layout(rng, counts, kind)
    R, used = int(off[-1]), [-(-n // page) for n in lens]
    pages = sum(used) + 2
    ids = rng.permutation(pages).astype(np.int32)
    table = np.full((len(counts), max(used) + 1), -7, dtype=np.int32)     # never read beyond the length
    at = 0
    for i, n in enumerate(used):
        table[i, :n] = ids[at:at + n]
        at += n
    draw = lambda *s: _bits(rng.standard_normal(s) * spread, dtype)
    return dict(q=draw(R, H, D), k=draw(R, KV, D), v=draw(R, KV, D), off=off, kc=draw(pages, page, KV, D),
                vc=draw(pages, page, KV, D), table=table, length=np.array(lens, dtype=np.int32), par=par, dtype=dtype,
                owner=owner)


def _call(vsv, c, chain=False, **kw):
    d = {k: to_dev(c[k]) for k in ("q", "k", "v", "off", "kc", "vc", "table", "length", "par")}
    d.update({k: kw.pop(k) for k in list(kw) if k in d})
    return vsv.tree_attention(d["q"], d["k"], d["v"], d["off"], d["kc"], d["vc"], d["table"], d["length"],
                              parents=None if chain else d["par"], return_lse=True, **kw)


def _check(out, lse, c, rows=None, scale=None):
    """Rows against the oracle, with the tolerances above."""
    dtype = c["dtype"]
    f = lambda a: oracle.bf16_bits_to_f64(a) if a.dtype == np.uint16 else a.astype(np.float64)
    R, H, D = c["q"].shape
    want, want_lse = oracle.tree_attention(c["q"], c["k"], c["v"], c["off"], c["kc"], c["vc"], c["table"], c["length"],
                                           c["par"], scale)
    mag_v = oracle.tree_attention(c["q"], c["k"], np.abs(f(c["v"])), c["off"], c["kc"], np.abs(f(c["vc"])), c["table"],
                                  c["length"], c["par"], scale)[0]
    sc = D ** -0.5 if scale is None else scale
    biggest = max(np.abs(f(c["k"])).max(), np.abs(f(c["kc"])).max())
    qk = np.abs(f(c["q"])).sum(2) * biggest * sc          # bounds sum |q k| and every score
    T = (c["length"].max(initial=0) + 64)
    e = 2 * D * 2.0 ** -24 * qk + 2.0 ** -21 * (1 + qk)
    h = 2.0 ** -8 if dtype == BF16 else 0.0
    half = 2.0 ** -8 if dtype == BF16 else 2.0 ** -24
    tol = (2 * e + h + T * 2.0 ** -23)[:, :, None] * mag_v + half * np.abs(want) + 1e-30
    got, got_lse = out.float().cpu().numpy().astype(np.float64), host(lse).astype(np.float64)
    rows = range(R) if rows is None else rows
    for r in rows:
        off = bool(np.any(~(np.abs(got[r] - want[r]) <= tol[r])))
        assert not off, (r, np.abs(got[r] - want[r]).max(), tol[r].min())
        off = bool(np.any(~(np.abs(got_lse[r] - want_lse[r]) <= e[r] + 2.0 ** -22 * (1 + np.abs(want_lse[r])))))
        assert not off, r


CASES = [
    # counts, lens, H, KV, D, page: every query block, single tokens, empty contexts, pages that end in a tile
    ([1], [0], 1, 1, 64, 16),
    ([1], [1], 2, 1, 128, 1),
    ([5], [300], 8, 2, 128, 16),
    ([3, 1, 64, 2], [17, 0, 255, 128], 4, 4, 64, 8),
    ([6] * 5, [31, 32, 33, 127, 640], 10, 2, 128, 32),
    ([2, 9, 0, 5], [1000, 3, 50, 129], 14, 2, 64, 128),
    ([50, 20], [257, 700], 10, 2, 128, 64),
    ([64, 64], [100, 65], 16, 2, 64, 2),
    ([1] * 300, [int(7 * i) % 130 for i in range(300)], 2, 1, 64, 16),
]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_attention_matches_the_definition(vsv, dtype, case):
    counts, lens, H, KV, D, page = CASES[case]
    c = _case(case, counts, lens, H, KV, D, page, dtype)
    print("attention case %d dtype=%d rows=%d" % (case, dtype, c["off"][-1]), flush=True)
    out, lse = _call(vsv, c)
    _check(out, lse, c)


@pytest.mark.parametrize("counts", [[2, 3], [20, 9], [40, 64]])
def test_head_dim_256(vsv, counts):
    c = _case(40, counts, [70, 333], 4, 2, 256, 16, BF16)
    print("attention D=256 %s" % counts, flush=True)
    _check(*_call(vsv, c), c)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_chains_without_parents(vsv, dtype):
    c = _case(41, [5, 64, 1], [40, 200, 9], 8, 2, 128, 16, dtype, "chain")
    out, lse = _call(vsv, c, chain=True)
    _check(out, lse, c)
    same, _ = _call(vsv, c)
    assert np.array_equal(host(same.float()), host(out.float()))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_long_contexts_are_cut_and_joined(vsv, dtype):
    # more pieces than a wave has lanes in one case: one head, one request
    c = _case(42, [3], [20000], 2, 1, 64, 64, dtype)
    print("attention long dtype=%d" % dtype, flush=True)
    _check(*_call(vsv, c), c)


def test_scores_that_keep_rising(vsv):
    # the reference moves at every tile, and far scores underflow
    c = _case(43, [4, 2], [900, 500], 2, 1, 64, 16, F32)
    for i in range(2):
        for t in range(int(c["length"][i])):
            c["kc"][c["table"][i, t // 16], t % 16] *= 0.02 * t
    _check(*_call(vsv, c, scale=0.7), c, scale=float(np.float32(0.7)))


def test_strides_of_one_projection_and_of_a_head_first_cache(vsv):
    import torch
    c = _case(44, [7, 3, 12], [90, 0, 33], 6, 2, 64, 16, BF16)
    q, k, v = [to_dev(c[n]) for n in ("q", "k", "v")]
    wide = torch.full((22, 6 + 2 + 2 + 1, 72), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, :6, :64], wide[:, 6:8, :64], wide[:, 8:10, :64] = q, k, v
    kc, vc = [to_dev(c[n]).permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3) for n in ("kc", "vc")]
    both = torch.stack((kc, vc), 1)
    out = torch.full((22, 6, 80), 3.0, dtype=torch.bfloat16, device="cuda")[:, :, 8:72]
    got, lse = _call(vsv, c, q=wide[:, :6, :64], k=wide[:, 6:8, :64], v=wide[:, 8:10, :64], kc=both[:, 0], vc=both[:, 1],
                     out=out)
    assert got.data_ptr() == out.data_ptr()
    _check(got, lse, c)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_what_a_row_does_not_see_cannot_reach_it(vsv, dtype):
    """NaN and infinities in rows off the path, in pages behind the length and
    in the tail of a page."""
    c = _case(45, [6, 64, 5], [37, 130, 0], 4, 2, 64, 16, dtype)
    clean = {k: c[k].copy() for k in ("k", "v", "kc", "vc")}
    nan, inf = _bits(np.array([np.nan]), dtype)[0], _bits(np.array([np.inf]), dtype)[0]
    # rows of request 1 that hang below row 3, and one row of request 0
    r0 = 6
    bad = {r0 + j for j in range(64) if 3 in oracle.path_of(c["par"][6:70], j)} | {2}
    for r in (r0 + 3, 2):
        c["k"][r], c["v"][r, :, ::2], c["v"][r, :, 1::2] = nan, inf, nan
    used = {int(p) for i in range(3) for p in c["table"][i, :-(-int(c["length"][i]) // 16)]}
    for p in range(c["kc"].shape[0]):
        if p not in used:
            c["kc"][p], c["vc"][p] = nan, inf
    for i, n in enumerate((37, 130)):
        p = c["table"][i, n // 16]
        c["kc"][p, n % 16:], c["vc"][p, n % 16:] = nan, nan
    sees = [r for r in range(75) if r not in bad and 2 not in ([] if r > 5 else oracle.path_of(c["par"][:6], r))]
    out, lse = _call(vsv, c)
    c2 = dict(c, **clean)
    _check(out, lse, c2, rows=sees)
    got = host(out.float())
    assert np.all(np.isnan(got[r0 + 3])) and np.all(np.isnan(got[2]))


def test_an_infinite_value_that_is_seen(vsv):
    c = _case(46, [3], [20], 1, 1, 64, 16, BF16)
    c["par"] = np.array([-1, 0, 0], dtype=np.int32)
    c["v"][1, 0, 5] = _bits(np.array([-np.inf]), BF16)[0]
    got = host(_call(vsv, c)[0].float())
    assert got[1, 0, 5] == -np.inf and np.all(np.isfinite(np.delete(got[1, 0], 5)))
    assert np.all(np.isfinite(got[0])) and np.all(np.isfinite(got[2]))


def test_padded_batches_leave_the_rest(vsv):
    import torch
    c = _case(47, [4, 2], [30, 60], 4, 2, 64, 16, F32)
    pad = lambda a: np.concatenate((a, np.full((5,) + a.shape[1:], np.nan, dtype=np.float32)))
    q, k, v = [to_dev(pad(c[n])) for n in ("q", "k", "v")]
    out = torch.full((11, 4, 64), 9.0, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    table = np.concatenate((c["table"], c["table"][:1] * 0))
    got, lse = _call(vsv, c, q=q, k=k, v=v, off=to_dev(np.array([0, 4, 6, 6], dtype=np.int32)), table=to_dev(table),
                     length=to_dev(np.array([30, 60, 5], dtype=np.int32)), out=out, error_flag=err,
                     par=to_dev(np.concatenate((c["par"], np.full(5, 99, dtype=np.int32)))))
    _check(got[:6], lse[:6], c)
    assert torch.all(out[6:] == 9.0) and int(err) == 0


def test_device_conditions(vsv):
    import torch
    def run(**kw):
        c = _case(48, [4, 6], [30, 60], 4, 2, 64, 16, F32)
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = torch.full((10, 4, 64), 9.0, device="cuda")
        _call(vsv, c, error_flag=err, out=out, **{k: to_dev(v) for k, v in kw.items()})
        return int(err), out
    i32 = lambda *a: np.array(a, dtype=np.int32)
    assert run()[0] == 0
    table = _case(48, [4, 6], [30, 60], 4, 2, 64, 16, F32)["table"]
    for bad in (10 ** 6, -1):
        t = table.copy()
        t[1, 2] = bad
        assert run(table=t)[0] == vsv.FLAG_PAGES
    for kw in (dict(length=i32(30, 16 * table.shape[1] + 1)), dict(length=i32(30, -1)), dict(off=i32(0, 4, 11)),
               dict(off=i32(0, 4, 2))):
        bits, out = run(**kw)
        assert bits == vsv.FLAG_LAYOUT
        assert torch.all(out[4:] == 9.0) and not torch.any(out[:4] == 9.0)
    assert run(par=i32(-1, 0, 0, 0, -1, 0, 2, 0, 0, 0))[0] == vsv.FLAG_LAYOUT


def test_dimensions_of_one(vsv):
    import torch
    c = _case(49, [1], [30], 1, 1, 64, 16, BF16)
    # strides of dimensions of one element may be anything
    odd = lambda t: torch.as_strided(t, t.shape, (3, 5, 1))
    q, k, v = [odd(to_dev(c[n])) for n in ("q", "k", "v")]
    _check(*_call(vsv, c, q=q, k=k, v=v), c)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_caches_beyond_32_bits(vsv, dtype):
    """Pages whose elements lie past 2^32: the cache is allocated whole and
    filled at the pages in use alone."""
    import torch
    page, KV, D, pages = 64, 4, 128, 2 ** 32 // (64 * 4 * 128) + 40
    c = _case(50, [3, 5], [100, 777], 8, KV, D, page, dtype)
    used = [(i, j) for i, n in enumerate(c["length"]) for j in range(-(-int(n) // page))]
    kc, vc = [torch.empty((pages, page, KV, D), dtype=torch.bfloat16 if dtype == BF16 else torch.float32, device="cuda")
              for _ in range(2)]
    table = np.full_like(c["table"], -7)
    small = [to_dev(c[n]) for n in ("kc", "vc")]
    for m, (i, j) in enumerate(used):
        table[i, j] = pages - 1 - 2 * m if m % 3 else m
        for big, s in zip((kc, vc), small):
            big[int(table[i, j])] = s[int(c["table"][i, j])]
    print("cache of %d elements dtype=%d" % (kc.numel(), dtype), flush=True)
    _check(*_call(vsv, c, kc=kc, vc=vc, table=to_dev(table)), c)
    del kc, vc
