"""Pins of the tree oracle: chains against the linear oracle, closed forms and
brute force. Needs no GPU."""
import itertools

import numpy as np

import oracle
import synth


def test_chains_match_the_linear_oracle():
    for key in ("tiny",):
        wl = synth.make(key)
        want = oracle.verify_greedy(wl.logits, wl.dtype, wl.V, wl.offsets, wl.owner, wl.drafts)
        parents = np.concatenate([np.arange(b - a) - 1 for a, b in zip(wl.offsets[:-1], wl.offsets[1:])])
        for par in (None, parents):
            got = oracle.verify_greedy_tree(wl.logits, wl.dtype, wl.V, wl.offsets, wl.drafts, par)
            n = int(want["out_offsets"][-1])
            for k in ("accepted_len", "next_token", "out_offsets", "row_token"):
                assert np.array_equal(got[k], want[k]), k
            assert np.array_equal(got["out_tokens"], want["out_tokens"][:n])
            rows = np.concatenate([wl.offsets[i] + np.arange(a + 1) for i, a in enumerate(want["accepted_len"])])
            assert np.array_equal(got["out_rows"], rows)


def test_every_tree_of_five_rows():
    # the accepted path is the longest one that follows the arg-maxes, and
    # the lowest rows among those
    V, rng = 3, np.random.default_rng(0)
    for parents in itertools.product((0,), (0, 1), (0, 1, 2), (0, 1, 2, 3)):
        par = np.array((-1,) + parents)
        drafts, token = rng.integers(0, V, 4), rng.integers(0, V, 5)
        logits = np.zeros((5, V), dtype=np.float32)
        logits[np.arange(5), token] = 1.0
        got = oracle.verify_greedy_tree(logits, oracle.F32, V, [0, 5], drafts, par)
        fits = [p for p in (oracle.path_of(par, j) for j in range(5))
                if all(drafts[b - 1] == token[a] for a, b in zip(p, p[1:]))]
        # children that carry the same token lead to the lowest one alone
        best = [0]
        while True:
            more = [p for p in fits if len(p) == len(best) + 1 and p[:-1] == best]
            if not more:
                break
            best = min(more)
        assert got["out_rows"].tolist() == best
        assert got["accepted_len"][0] == len(best) - 1 and got["next_token"][0] == token[best[-1]]


def test_adjustments():
    x = np.array([2.0, -2.0, 1.0, 0.5, -1.0])
    y = oracle.adjust_row(x, [1], [0, 0, 4], repetition=2.0, frequency=0.25, presence=1.0,
                          bias=[(3, 1.0), (3, -2.0), (2, 4.0)], allowed=[1, 1, 0, 1, 1])
    assert np.allclose(y, [1.0 - 0.5 - 1.0, -4.0, -np.inf, -1.5, -2.0 - 0.25 - 1.0])


def test_pages_are_neither_lost_nor_shared():
    rng = np.random.default_rng(1)
    B, W, page, pool = 6, 8, 4, 30
    table = np.full((B, W), -1, dtype=np.int32)
    free = np.arange(pool, dtype=np.int32)
    rng.shuffle(free)
    count, held, length = pool, np.zeros(B, dtype=np.int32), np.zeros(B, dtype=np.int32)
    for _ in range(40):
        rows = rng.integers(0, 9, B)
        over = rng.random(B) < 0.25
        length = np.where(over, 0, length).astype(np.int32)
        rows = np.where(over | (length + rows > W * page), 0, rows)
        off = np.concatenate(([0], np.cumsum(rows)))
        out = oracle.plan_pages(table, held, length, off, free, count, page, off[-1] + 2)
        table, free, count = out["block_table"], out["free_pages"], int(out["free_count"][0])
        held, length = out["held"], out["length"]
        ids = [int(p) for i in range(B) for p in table[i, :held[i]]] + free[:count].tolist()
        assert sorted(ids) == list(range(pool))
        used = out["slot"][out["slot"] >= 0]
        assert len(set(used.tolist())) == len(used)
        assert out["short"] or np.array_equal(held, -(-length // page))


def test_attention_closed_forms():
    rng = np.random.default_rng(2)
    k = np.zeros((3, 1, 8), dtype=np.float32)        # equal scores: means of the values
    v = rng.standard_normal((3, 1, 8)).astype(np.float32)
    q = rng.standard_normal((3, 2, 8)).astype(np.float32)
    kc = np.zeros((2, 4, 1, 8), dtype=np.float32)
    vc = rng.standard_normal((2, 4, 1, 8)).astype(np.float32)
    par = np.array([-1, 0, 0])
    out, lse = oracle.tree_attention(q, k, v, [0, 3], kc, vc, np.array([[1, 0]]), [5], par)
    ctx = np.concatenate((vc[1, :, 0], vc[0, :1, 0]))
    for r, own in enumerate(([0], [0, 1], [0, 2])):
        want = np.concatenate((ctx, v[own, 0])).mean(0)
        assert np.allclose(out[r], want) and np.allclose(lse[r], np.log(5 + len(own)))
