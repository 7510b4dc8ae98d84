"""Attention of draft trees where a workgroup takes many tiles: every
instantiation at batches that fill the chip several times over, spans that
look their pages up again, scores that pass the reference at every step.

Tolerances as in test_gpu_attention.py, with |q k| bounded by the product of
the norms, and with the longest chain of additions in the place of all tokens:
a span's, at most 2 * (tokens of the batch's items) / workgroups + two tiles,
and 512 pieces."""
import numpy as np
import pytest

from tests.tree_cases import layout
from tests.workloads import cuda_or_skip, to_dev

pytestmark = pytest.mark.gpu

# query heads a key head, rows of a request: blocks of 16, 32, 64, 128 and 256 queries
BLOCKS = {16: (2, 2, 8), 32: (5, 4, 7), 64: (8, 4, 8), 128: (8, 9, 16), 256: (8, 15, 36)}
KERNELS = [(t, d, m) for t in ("float32", "bfloat16") for d in (64, 128, 256) for m in BLOCKS
           if (t == "bfloat16" or d < 256) and (d < 256 or m < 256)]


@pytest.fixture(scope="module")
def vsv():
    cuda_or_skip()
    import draft_token_verification_packed_amd as m
    m.lib()
    return m


def _case(seed, dtype, D, block, KV, B, lens, page, grow=0.0, sharp=1.0):
    import torch
    rng = np.random.default_rng(seed)
    g = torch.Generator(device="cuda").manual_seed(seed)
    G, lo, hi = BLOCKS[block]
    dt = getattr(torch, dtype)
    counts = rng.integers(lo, hi + 1, B)
    off, _, par = layout(rng, counts)
    length = rng.integers(lens[0], lens[1] + 1, B).astype(np.int32)
    used = -(-length // page)
    pages = int(used.sum()) + 3
    ids = rng.permutation(pages).astype(np.int32)
    table = np.full((B, int(used.max()) + 1), -7, dtype=np.int32)
    at = 0
    for i, n in enumerate(used):
        table[i, :n] = ids[at:at + n]
        at += n
    f = lambda *s: torch.randn(*s, device="cuda", generator=g)
    R = int(off[-1])
    c = dict(q=(f(R, G * KV, D) * sharp).to(dt), k=f(R, KV, D).to(dt), v=f(R, KV, D).to(dt),
             kc=f(pages, page, KV, D).to(dt), vc=f(pages, page, KV, D).to(dt), off=off, par=par, length=length, table=table,
             dev=[to_dev(a) for a in (off, table, length, par)])
    if grow:
        for i, n in enumerate(length):
            t = torch.arange(int(n), device="cuda")
            where = c["dev"][1][i].long()[t // page], t % page
            c["kc"][where] = (c["kc"][where].float() * (grow * t)[:, None, None]).to(dt)
    return c


def _call(vsv, c):
    off, table, length, par = c["dev"]
    return vsv.tree_attention(c["q"], c["k"], c["v"], off, c["kc"], c["vc"], table, length, par, return_lse=True)


def _check(c, out, lse, requests):
    """Rows of `requests` against sums in 64 bits."""
    import torch
    R, H, D = c["q"].shape
    KV, page = c["k"].shape[1], c["kc"].shape[1]
    G, scale, bf16 = H // KV, D ** -0.5, out.dtype is torch.bfloat16
    half, weight = (2.0 ** -8, 2.0 ** -8) if bf16 else (2.0 ** -24, 0.0)
    n_all = c["length"].astype(np.int64) + np.diff(c["off"])
    chain = 2 * KV * int(n_all.sum()) * (1 + G * 36 // 256) / 256 + 256 + 512
    for i in requests:
        r0, r1, n = int(c["off"][i]), int(c["off"][i + 1]), int(c["length"][i])
        t = torch.arange(n, device="cuda")
        where = c["dev"][1][i].long()[t // page], t % page
        sees = np.eye(r1 - r0, dtype=bool)
        for j in range(1, r1 - r0):
            sees[j] |= sees[c["par"][r0 + j]]
        sees = torch.cat((torch.ones(r1 - r0, n, dtype=torch.bool, device="cuda"), to_dev(sees)), 1)
        for h in range(KV):
            keys = torch.cat((c["kc"][where[0], where[1], h], c["k"][r0:r1, h])).double()
            values = torch.cat((c["vc"][where[0], where[1], h], c["v"][r0:r1, h])).double()
            x = c["q"][r0:r1, h * G:(h + 1) * G].double().reshape(-1, D)
            s = torch.mm(x, keys.t().contiguous()) * scale
            s.masked_fill_(~sees.repeat_interleave(G, 0), -np.inf)
            want_lse = torch.logsumexp(s, 1)
            p = torch.exp(s - want_lse[:, None])
            want, mag = torch.mm(p, values), torch.mm(p, values.abs())
            qk = x.norm(dim=1) * keys.norm(dim=1).max() * scale
            e = 2 * D * 2.0 ** -24 * qk + 2.0 ** -21 * (1 + qk)
            tol = (2 * e + weight + min(chain, n + 64) * 2.0 ** -23)[:, None] * mag + half * want.abs() + 1e-30
            got = out[r0:r1, h * G:(h + 1) * G].double().reshape(-1, D)
            err = (got - want).abs()
            assert bool((err <= tol).all()), (i, h, float((err / tol).max()))
            got = lse[r0:r1, h * G:(h + 1) * G].double().reshape(-1)
            assert bool(((got - want_lse).abs() <= e + 2.0 ** -22 * (1 + want_lse.abs())).all()), (i, h)


@pytest.mark.parametrize("dtype,D,block", KERNELS)
def test_batches_that_fill_the_chip_several_times(vsv, dtype, D, block):
    B, lens = (96, (0, 1100)) if block < 256 else (48, (0, 3000))
    c = _case(D + block, dtype, D, block, 8, B, lens, 16)
    print("attention %s D=%d block=%d" % (dtype, D, block), flush=True)
    out, lse = _call(vsv, c)
    _check(c, out, lse, range(0, B, 5))
    # the order of workgroups and waves cannot show
    for _ in range(3):
        again, lse2 = _call(vsv, c)
        assert bool((out == again).all()) and bool((lse == lse2).all())


@pytest.mark.parametrize("dtype,D,block", [k for k in KERNELS if k[1] in (64, 128)])
def test_scores_that_pass_the_reference_at_every_step(vsv, dtype, D, block):
    c = _case(3 * D + block, dtype, D, block, 8, 64 if block < 256 else 24, (500, 1500), 32, grow=0.05)
    print("attention rising %s D=%d block=%d" % (dtype, D, block), flush=True)
    _check(c, *_call(vsv, c), range(0, 24, 5))


@pytest.mark.parametrize("dtype,block,n", [("float32", 16, 700000), ("float32", 64, 600000), ("float32", 256, 300000),
                                           ("bfloat16", 32, 700000), ("bfloat16", 256, 300000)])
def test_spans_that_look_their_pages_up_again(vsv, dtype, block, n):
    # pages of one token, more than 1023 of them in every span
    c = _case(block, dtype, 64, block, 1, 1, (n, n), 1, sharp=3.0)
    print("attention pages %s block=%d" % (dtype, block), flush=True)
    _check(c, *_call(vsv, c), [0])


def test_mixed_batches(vsv):
    """One tree of 64 rows and long requests among single rows: items of every
    length in one list."""
    import torch
    c = _case(9, "bfloat16", 128, 32, 4, 60, (0, 300), 16)
    rng = np.random.default_rng(1)
    counts = np.ones(60, dtype=np.int64)
    counts[7], counts[30] = 64, 0
    off, _, par = layout(rng, counts)
    R = int(off[-1])
    g = torch.Generator(device="cuda").manual_seed(5)
    for k, heads in (("q", 20), ("k", 4), ("v", 4)):
        c[k] = torch.randn(R, heads, 128, device="cuda", generator=g).to(torch.bfloat16)
    c.update(off=off, par=par)
    c["dev"][0], c["dev"][3] = to_dev(off), to_dev(par)
    _check(c, *_call(vsv, c), [0, 6, 7, 8, 29, 31, 59])


def _plain(seed, counts, lens, H, KV, D, page, dtype):
    """A batch of given rows and lengths."""
    import torch
    rng = np.random.default_rng(seed)
    c = _case(seed, dtype, D, 16, KV, len(counts), (0, 1), page)
    off, _, par = layout(rng, counts)
    length = np.array(lens, dtype=np.int32)
    used = -(-length // page)
    pages = int(used.sum()) + 2
    ids, at = rng.permutation(pages).astype(np.int32), 0
    table = np.full((len(counts), int(used.max()) + 1), -7, dtype=np.int32)
    for i, n in enumerate(used):
        table[i, :n] = ids[at:at + n]
        at += n
    g = torch.Generator(device="cuda").manual_seed(seed)
    f = lambda *s: torch.randn(*s, device="cuda", generator=g).to(getattr(torch, dtype))
    R = int(off[-1])
    c.update(q=f(R, H, D), k=f(R, KV, D), v=f(R, KV, D), kc=f(pages, page, KV, D), vc=f(pages, page, KV, D), off=off, par=par,
             length=length, table=table, dev=[to_dev(a) for a in (off, table, length, par)])
    return c


@pytest.mark.parametrize("dtype,counts,lens,H,KV,page", [
    ("bfloat16", [64, 3], [2000, 700], 128, 1, 16),          # one key head: 8192 queries in many blocks
    ("float32", [20, 64], [300, 1000], 96, 1, 32),
    ("bfloat16", [5, 2, 9], [5000, 70000, 0], 10, 2, 65536),  # pages longer than a context
    ("float32", [1, 4], [70000, 3], 4, 2, 131072),
])
def test_shapes_at_the_ends(vsv, dtype, counts, lens, H, KV, page):
    c = _plain(3, counts, lens, H, KV, 64, page, dtype)
    print("attention ends %s %s" % (dtype, counts), flush=True)
    _check(c, *_call(vsv, c), range(len(counts)))


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_thousands_of_requests(vsv, dtype):
    # more requests than a workgroup has threads, many of them without rows
    rng = np.random.default_rng(4)
    counts = rng.integers(0, 4, 9000)
    counts[5000:7000] = 0
    lens = rng.integers(0, 60, 9000)
    c = _plain(5, counts, lens, 4, 2, 64, 16, dtype)
    _check(c, *_call(vsv, c), [int(i) for i in np.flatnonzero(counts)[::211]])
