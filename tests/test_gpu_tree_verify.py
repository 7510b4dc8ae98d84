"""Greedy verification of trees against the oracle. Tokens, lengths and rows
are exact; log-sum-exps hold to the tolerance of linear verification."""
import numpy as np
import pytest

import oracle
import synth
from tests.tree_cases import layout
from tests.workloads import assert_lse_close, assert_same, cuda_or_skip, host, oracle_of, to_dev, upload

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def vsv():
    cuda_or_skip()
    import draft_token_verification_packed_amd as m
    m.lib()
    return m


def _batch(seed, counts, V, dtype, kind="wide", pad=0):
    """Rows whose arg-max is mostly a child's draft, few distinct drafts (so
    that siblings share tokens), and ties inside rows."""
    rng = np.random.default_rng(seed)
    off, owner, par = layout(rng, counts, kind)
    R, B = int(off[-1]), len(counts)
    x = np.round(rng.standard_normal((R, V)) * 2).astype(np.float32)
    drafts = rng.integers(0, min(V, 5), R - B).astype(np.int32)
    for r in range(R):
        i = owner[r]
        kids = [c for c in range(r + 1, off[i + 1]) if off[i] + par[c] == r]
        if kids and rng.random() < 0.85:
            x[r, drafts[rng.choice(kids) - i - 1]] = 60.0
    store = np.full((R, V + pad), np.nan, dtype=np.float32)
    store[:, :V] = x
    return off, owner, par, drafts, synth.f32_to_bf16_bits(store) if dtype == oracle.BF16 else store


def _check(out, ref, R):
    n = int(ref["out_offsets"][-1])
    for k in ("accepted_len", "next_token", "out_offsets", "row_token"):
        assert np.array_equal(host(out[k]), ref[k]), k
    for k in ("out_tokens", "out_rows"):
        got = host(out[k])
        assert np.array_equal(got[:n], ref[k]), k
        assert np.all(got[n:] == -1), k
    assert_lse_close(host(out["row_lse"]), ref["row_lse"])
    assert int(host(out["error_flag"])[0]) == 0


@pytest.mark.parametrize("dtype", [oracle.F32, oracle.BF16])
@pytest.mark.parametrize("counts,V,kind,pad", [
    ([1], 1, "wide", 0), ([2, 1, 64], 33, "wide", 3), ([64] * 5, 1000, "chain", 0), ([5] * 40, 257, "wide", 1),
    ([7, 50, 1, 33, 64, 2], 4099, "wide", 5), ([3] * 300 + [64] * 30, 64, "wide", 0), ([64] * 70, 40, "wide", 0),
])
def test_trees_match_the_oracle(vsv, dtype, counts, V, kind, pad):
    off, owner, par, drafts, store = _batch(len(counts) + V, counts, V, dtype, kind, pad)
    print("tree verify %d requests V=%d dtype=%d %s" % (len(counts), V, dtype, kind), flush=True)
    ref = oracle.verify_greedy_tree(store, dtype, V, off, drafts, par)
    d = [to_dev(a) for a in (store, off, owner, drafts, par)]
    _check(vsv.verify_greedy_tree(*d, vocab=V), ref, int(off[-1]))
    if kind == "chain":
        _check(vsv.verify_greedy_tree(*d[:4], None, vocab=V), ref, int(off[-1]))


def test_chains_match_linear_verification(vsv):
    wl = synth.make("eagle", B=16)
    d = upload(wl)
    out = vsv.verify_greedy_tree(d["logits"], d["offsets"], d["owner"], d["drafts"], None, vocab=wl.V)
    assert_same(out, oracle_of(wl))


def test_device_conditions(vsv):
    off, owner, par, drafts, store = _batch(5, [4, 6, 3], 50, oracle.F32)
    d = [to_dev(a) for a in (store, off, owner, drafts)]
    bad = par.copy()
    bad[5], bad[6] = 3, -1             # no earlier rows of their request
    out = vsv.verify_greedy_tree(*d, to_dev(bad))
    assert int(host(out["error_flag"])[0]) == vsv.FLAG_LAYOUT
    far = drafts.copy()
    far[:] = 50
    out = vsv.verify_greedy_tree(*d[:3], to_dev(far), to_dev(par))
    assert int(host(out["error_flag"])[0]) == vsv.FLAG_TOKEN
    assert host(out["accepted_len"]).tolist() == [0, 0, 0]
    # more rows than a tree may have, offsets that fall, and an owner of no request
    counts = [65, 2]
    o2, w2, p2 = layout(np.random.default_rng(0), counts)
    x = np.zeros((67, 8), dtype=np.float32)
    out = vsv.verify_greedy_tree(to_dev(x), to_dev(o2), to_dev(w2), to_dev(np.zeros(65, dtype=np.int32)), to_dev(p2))
    assert int(host(out["error_flag"])[0]) & vsv.FLAG_LAYOUT
    fall = off.copy()
    fall[1], fall[2] = 9, 4
    for o, w in ((fall, owner), (off, np.full_like(owner, 7))):
        out = vsv.verify_greedy_tree(d[0], to_dev(o), to_dev(w), d[3], to_dev(par))
        assert int(host(out["error_flag"])[0]) & vsv.FLAG_LAYOUT
    # the workspace serves the next call
    ref = oracle.verify_greedy_tree(store, oracle.F32, 50, off, drafts, par)
    _check(vsv.verify_greedy_tree(*d, to_dev(par)), ref, int(off[-1]))
