"""Random batches through the tree operators: shapes, alignment, strides, types
and options drawn per case, against the oracle with the tolerances of the
operators' own tests."""
import numpy as np
import pytest

import oracle
import synth
from tests import test_gpu_adjust, test_gpu_attention, test_gpu_pages, test_gpu_tree_verify
from tests.workloads import cuda_or_skip, host, to_dev

pytestmark = pytest.mark.gpu

SEEDS = 40


@pytest.fixture(scope="module")
def vsv():
    cuda_or_skip()
    import draft_token_verification_packed_amd as m
    m.lib()
    return m


def _log(rng, lo, hi):
    return int(round(np.exp(rng.uniform(np.log(lo), np.log(hi)))))


def _counts(rng, most, rows):
    n = _log(rng, 1, most)
    hi = _log(rng, 1, rows)
    return [int(c) for c in rng.integers(1, hi + 1, n)]


def _shifted(a, shift, pad):
    """`a` as rows of a wider matrix that starts `shift` elements behind an
    aligned address."""
    import torch
    t = to_dev(a)
    wide = torch.zeros((t.shape[0] + 1) * (t.shape[1] + pad) + shift, dtype=t.dtype, device="cuda")
    view = wide[shift:shift + t.shape[0] * (t.shape[1] + pad)].view(t.shape[0], -1)[:, :t.shape[1]]
    view.copy_(t)
    return view


def adjust(vsv, seed):
    rng = np.random.default_rng(seed)
    dtype, kind = (oracle.F32, oracle.BF16)[rng.integers(0, 2)], ("chain", "wide")[rng.integers(0, 2)]
    counts = _counts(rng, 24, 64)
    V = _log(rng, 1, 6000)
    full = int(rng.integers(0, 4))
    c = test_gpu_adjust._case(seed, counts, V, dtype, kind, int(rng.integers(0, 9)), H=_log(rng, 1, 400),
                              bias=int(rng.integers(0, 12)), masked=float(rng.random()), full=full,
                              tokens=max(1, int(V * rng.random())))
    drop = [n for n in ("history", "bias", "mask", "penalties") if rng.random() < 0.2]
    kw = {}
    for n in drop:
        kw.update(dict(history=dict(history=None, history_len=None, prompt_len=None),
                       bias=dict(bias_offsets=None, bias_tokens=None, bias_values=None), mask=dict(mask=None, mask_index=None),
                       penalties=dict(repetition=None, frequency=None, presence=None))[n])
    chain = kind == "chain" and rng.random() < 0.5 and not full
    x = _shifted(c["store"], int(rng.integers(0, 9)), 0)
    got = test_gpu_adjust._call(vsv, c, store=x, chain=chain, **kw)
    test_gpu_adjust._check(got, c, drop)
    same = test_gpu_adjust._call(vsv, c, store=x, chain=chain, out=x, **kw)
    assert np.array_equal(host(same.float())[:c["R"]], host(got.float())[:c["R"]], equal_nan=True)


def verify(vsv, seed):
    rng = np.random.default_rng(seed)
    dtype = (oracle.F32, oracle.BF16)[rng.integers(0, 2)]
    counts = _counts(rng, 120, 64)
    V, kind = _log(rng, 1, 5000), ("chain", "wide")[rng.integers(0, 2)]
    off, owner, par, drafts, store = test_gpu_tree_verify._batch(seed, counts, V, dtype, kind, int(rng.integers(0, 9)))
    ref = oracle.verify_greedy_tree(store, dtype, V, off, drafts, par)
    x = _shifted(store, int(rng.integers(0, 9)), 0)
    out = vsv.verify_greedy_tree(x, to_dev(off), to_dev(owner), to_dev(drafts), to_dev(par), vocab=V)
    test_gpu_tree_verify._check(out, ref, int(off[-1]))


def pages(vsv, seed):
    rng = np.random.default_rng(seed)
    B = _log(rng, 1, 3000)
    state = test_gpu_pages._state(rng, B, _log(rng, 1, 128), _log(rng, 1, 500), _log(rng, 1, 60), _log(rng, 1, 4 * B + 1))
    test_gpu_pages._check(vsv, state, int(state[3][-1]) + int(rng.integers(0, 50)))


def attention(vsv, seed):
    rng = np.random.default_rng(seed)
    dtype = (oracle.F32, oracle.BF16)[rng.integers(0, 2)]
    D = int(rng.choice((64, 128, 256) if dtype == oracle.BF16 else (64, 128)))
    kv, group = _log(rng, 1, 4), _log(rng, 1, 9)
    counts = _counts(rng, 6, 64 if group < 4 else 24)
    lens = [int(n) for n in rng.integers(0, _log(rng, 1, 500) + 1, len(counts))]
    kind = ("chain", "wide")[rng.integers(0, 2)]
    c = test_gpu_attention._case(seed, counts, lens, kv * group, kv, D, 1 << int(rng.integers(0, 8)), dtype, kind,
                                 float(rng.choice((0.3, 1.0, 1.5))))
    if rng.random() < 0.3:      # requests without rows, anywhere
        at = int(rng.integers(0, len(counts) + 1))
        for n, v in (("off", c["off"][at]), ("length", int(rng.integers(0, c["length"].max() + 1)))):
            c[n] = np.insert(c[n], at, v).astype(np.int32)
        c["table"] = np.insert(c["table"], at, 0, axis=0)
    out, lse = test_gpu_attention._call(vsv, c, chain=kind == "chain" and rng.random() < 0.5)
    test_gpu_attention._check(out, lse, c)


@pytest.mark.parametrize("run", [adjust, verify, pages, attention])
def test_random_batches(vsv, run):
    for seed in range(SEEDS):
        try:
            run(vsv, seed)
        except AssertionError as e:
            raise AssertionError("%s seed %d" % (run.__name__, seed)) from e
