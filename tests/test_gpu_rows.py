"""The row operators next to verification against their float64 definition:
drawn tokens, top logits, distillation and its gradient.

Tolerances of the float outputs. A draw's log-probability and log-sum-exp
come from sums within 1e-10 and are rounded once: |v| 2^-24, 1e-9 beside it.
Elsewhere the row's sum is one of float exponentials: exp2 within 2^-23, its
argument x log2(e) / T rounded (2^-24 of the |x - m| / T < 8 that holds the
weight) and the scale rounded once for the row (2^-24 of the largest |x| / T):
together below D = 2^-22 (1 + max|x| / T), for a sum over a part of the row
too. A loss is that error times masses that add up to one, twice where the
rest is a cell of its own. A gradient's element is q times a difference of
two numbers of size M and t_r / q_r, so its error is below
4 D q (M + t_r / q_r) weight / T, and half a step of its type for the one
rounding."""
import math

import numpy as np
import pytest

import oracle
from tests.row_cases import BF16, F32, KINDS, largest, row_values, rows_f64, store_rows
from tests.workloads import cuda_or_skip, host, to_dev

pytestmark = pytest.mark.gpu

HALF = {F32: 2.0 ** -24, BF16: 2.0 ** -8}


@pytest.fixture(scope="module")
def vsv():
    cuda_or_skip()
    import draft_token_verification_packed_amd as m
    m.lib()
    return m


def _store(seed, n, V, dtype, kinds, pad, shift, sigma=2.5):
    rng = np.random.default_rng(seed)
    rows = [row_values(rng, kinds[r % len(kinds)], V, dtype, sigma) for r in range(n)]
    store = store_rows(rows, dtype, pad, shift)
    return rng, to_dev(store)[:, shift:], rows_f64(store, dtype, V, shift)


# ------------------------------------------------------------------- draws

def _params(rng, n, V):
    T = rng.choice([0.0, 0.05, 0.5, 1.0, 1.0, 2.0, 30.0], size=n).astype(np.float32)
    k = rng.choice([0, 0, -1, 1, 2, 50, V - 1, V, V + 5], size=n).astype(np.int32)
    p = rng.choice([1.0, 1.0, 0.95, 0.5, 0.01], size=n).astype(np.float32)
    mp = rng.choice([0.0, 0.0, 1e-4, 0.1, 1.0], size=n).astype(np.float32)
    u = rng.random(n, dtype=np.float32)
    u[::7] = 0.0
    u[3::7] = np.float32(1 - 2.0 ** -24)
    return T, k, p, mp, u


def _check_draws(out, xs, T, k, p, mp, u):
    tok, lp, lse = host(out["token"]), host(out["logprob"]), host(out["lse"])
    for r, x in enumerate(xs):
        t, want_lp, want_lse = oracle.draw_row(x, float(T[r]), int(k[r]), float(p[r]), float(mp[r]), float(u[r]))
        at = (r, float(T[r]), int(k[r]), float(p[r]), float(mp[r]), float(u[r]))
        assert int(tok[r]) == t, (at, int(tok[r]), t)
        assert abs(lp[r] - want_lp) <= 2.0 ** -24 * abs(want_lp) + 1e-9, (at, lp[r], want_lp)
        assert abs(lse[r] - want_lse) <= 2.0 ** -24 * abs(want_lse) + 1e-9, (at, lse[r], want_lse)
    assert int(host(out["error_flag"])[0]) == 0


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("V,pad,shift", [(1, 0, 0), (2, 1, 1), (5, 3, 0), (63, 0, 1), (64, 0, 0), (1000, 1, 3),
                                         (4099, 0, 0), (4096, 0, 0), (20000, 7, 1)])
def test_draws(vsv, dtype, V, pad, shift):
    n = 96 if V < 10000 else 48
    rng, x, xs = _store(100 + V, n, V, dtype, KINDS, pad, shift)
    a = _params(rng, n, V)
    print("draws V=%d dtype=%d" % (V, dtype), flush=True)
    _check_draws(vsv.sample_rows(x, *[to_dev(q) for q in a], vocab=V), xs, *a)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("V,pad,shift", [(152064, 0, 0), (70001, 3, 1)])
def test_draws_over_a_full_vocabulary(vsv, dtype, V, pad, shift):
    # few long rows: each is cut into parts
    n = 24
    rng, x, xs = _store(7, n, V, dtype, ("plain", "spikes", "masked", "ties", "equal", "one_left", "lowest"), pad, shift)
    a = _params(rng, n, V)
    a[0][a[0] == 0] = 1.0
    _check_draws(vsv.sample_rows(x, *[to_dev(q) for q in a], vocab=V), xs, *a)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_draws_of_many_long_rows(vsv, dtype):
    # enough rows that each is one workgroup's
    import torch
    m, n, V = 4, 520, 70001
    rng, x, xs = _store(17, m, V, dtype, ("plain", "spikes", "ties", "masked"), 1, 0)
    x = x[torch.arange(n, device="cuda") % m].contiguous()
    a = _params(rng, n, V)
    _check_draws(vsv.sample_rows(x, *[to_dev(q) for q in a], vocab=V), [xs[r % m] for r in range(n)], *a)


def test_every_token_of_a_law_is_reached(vsv):
    # one row's law, walked by evenly spread numbers: both ends and every border
    V, n = 300, 4096
    rng = np.random.default_rng(3)
    row = row_values(rng, "ties", V, F32)
    store = store_rows([row] * n, F32)
    u = ((np.arange(n) + 0.5) / n).astype(np.float32)
    full = lambda v, t: np.full(n, v, dtype=t)
    a = (full(1.0, np.float32), full(0, np.int32), full(0.9, np.float32), full(0.0, np.float32), u)
    _check_draws(vsv.sample_rows(to_dev(store), *[to_dev(q) for q in a]), [row.astype(np.float64)] * n, *a)


def test_draws_agree_with_sampled_verification(vsv):
    # the same law and the same numbers: one request per row and no drafts
    n, V = 64, 4099
    rng, x, _ = _store(11, n, V, F32, ("plain", "spikes"), 0, 0)
    T = rng.choice([0.0, 0.7, 1.0], size=n).astype(np.float32)
    k = rng.choice([0, 50], size=n).astype(np.int32)
    p = rng.choice([1.0, 0.9], size=n).astype(np.float32)
    mp = rng.choice([0.0, 0.05], size=n).astype(np.float32)
    u = np.array([oracle.row_uniform(5, i, 0, 9) for i in range(n)], dtype=np.float32)
    par = [to_dev(q) for q in (T, k, p, mp)]
    off, own = to_dev(np.arange(n + 1, dtype=np.int32)), to_dev(np.arange(n, dtype=np.int32))
    ref = vsv.verify_sampled(x, off, own, None, *par, seed=5, offset=9)
    out = vsv.sample_rows(x, *par, to_dev(u))
    assert np.array_equal(host(out["token"]), host(ref["row_token"]))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_a_lone_survivor_is_certain(vsv, dtype):
    # whatever leaves one token, its log-probability is 0 and not a rounding
    n, V = 40, 4099
    rng, x, _ = _store(19, n, V, dtype, ("plain", "spikes", "wide"), 0, 0)
    f = lambda v: to_dev(np.full(n, v, dtype=np.float32))
    T, u = to_dev(rng.uniform(0.3, 2.0, n).astype(np.float32)), to_dev(rng.random(n, dtype=np.float32))
    one, off = to_dev(np.ones(n, dtype=np.int32)), to_dev(np.zeros(n, dtype=np.int32))
    for k, p, mp in ((one, 1.0, 0.0), (one, 0.9, 0.3), (off, 1e-6, 0.0), (one, 1.0, 0.05)):
        out = vsv.sample_rows(x, T, k, f(p), f(mp), u)
        assert not np.any(host(out["logprob"]))


def test_draw_flags(vsv):
    import torch
    V = 130
    rng, x, _ = _store(5, 8, V, F32, ("plain",), 0, 0)
    one, zero = torch.ones(8, device="cuda"), torch.zeros(8, device="cuda")
    k0 = torch.zeros(8, dtype=torch.int32, device="cuda")
    half = one * 0.5

    def flag(x=x, T=one, p=one, mp=zero, u=half):
        out = vsv.sample_rows(x, T, k0, p, mp, u)
        t = host(out["token"])
        assert np.all((t >= 0) & (t < V))
        return int(host(out["error_flag"])[0])

    def at(base, v):
        b = base.clone()
        b.view(-1)[3] = v
        return b

    assert flag() == 0
    for bad in (-1.0, math.inf, math.nan):
        assert flag(T=at(one, bad)) == vsv.FLAG_PARAMS
    for bad in (0.0, 1.5, math.nan):
        assert flag(p=at(one, bad)) == vsv.FLAG_PARAMS
    for bad in (-0.1, 1.1, math.nan):
        assert flag(mp=at(zero, bad)) == vsv.FLAG_PARAMS
        assert flag(u=at(half, bad)) == vsv.FLAG_PARAMS
    assert flag(u=at(half, 1.0)) == vsv.FLAG_PARAMS
    for bad in (math.nan, math.inf):
        assert flag(x=at(x, bad)) == vsv.FLAG_LOGITS
    none = x.clone()
    none[2] = -math.inf
    assert flag(x=none) == vsv.FLAG_LOGITS


# --------------------------------------------------------------- top logits

@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("V,k,pad,shift,T", [(1, 1, 0, 0, 1.0), (5, 5, 2, 1, 1.0), (64, 3, 0, 0, 0.5), (300, 256, 1, 1, 1.0),
                                             (1024, 8, 0, 0, 1.0), (4099, 64, 5, 3, 2.0), (20011, 256, 2, 0, 0.7),
                                             (152064, 1, 0, 0, 1.0), (152064, 100, 0, 0, 1.0)])
def test_top_logits(vsv, dtype, V, k, pad, shift, T):
    kinds = ("plain", "ties", "masked", "equal", "spikes", "one_left", "wide", "lowest")
    n = 24 if V < 100000 else 10
    rng, x, xs = _store(40 + V + k, n, V, dtype, kinds, pad, shift)
    print("top V=%d k=%d dtype=%d" % (V, k, dtype), flush=True)
    out = vsv.top_logits(x, k, temperature=T, vocab=V)
    v, ids, lse = host(out["values"]), host(out["ids"]), host(out["lse"])
    for r, xr in enumerate(xs):
        want_v, want_ids, want_lse = oracle.top_row(xr, k, T)
        assert np.array_equal(ids[r], want_ids), (r, kinds[r % 8])
        assert np.array_equal(v[r], want_v.astype(np.float32)), r
        tol = 2.0 ** -22 * (1 + largest(xr, T)) + 2.0 ** -24 * abs(want_lse)
        assert abs(lse[r] - want_lse) <= tol, (r, kinds[r % 8], lse[r], want_lse)
    assert int(host(out["error_flag"])[0]) == 0


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("order", ["rising", "falling", "blocks", "stride"])
@pytest.mark.parametrize("V,k", [(30000, 200), (30000, 40), (90001, 130)])
def test_top_logits_of_ordered_rows(vsv, dtype, order, V, k):
    # the largest elements late, early, together, or all in the same lanes;
    # rows taken whole and in parts
    x = np.sort(np.random.default_rng(8).standard_normal(V).astype(np.float32) * 3)
    if order == "falling":
        x = x[::-1].copy()
    elif order == "blocks":
        x = np.concatenate((x[V // 3:V // 2], x[V // 2:], x[:V // 3]))
    elif order == "stride":
        x = x.copy()
        big = np.sort(np.random.default_rng(9).random(2000).astype(np.float32)) + 20
        at = (np.arange(2000) % 4) + (np.arange(2000) // 4 % 7) * 4096 + np.arange(2000) // 28 * 8
        x[at % V] = big
    store = store_rows([x] * 3, dtype)
    out = vsv.top_logits(to_dev(store), k)
    for r, xr in enumerate(rows_f64(store, dtype, V, 0)):
        _, ids, _ = oracle.top_row(xr, k)
        assert np.array_equal(host(out["ids"])[r], ids)


def test_top_logits_flags(vsv):
    V = 700
    rng, x, _ = _store(6, 4, V, F32, ("plain",), 0, 0)
    for bad in (math.nan, math.inf):
        y = x.clone()
        y[1, 77] = bad
        out = vsv.top_logits(y, 9)
        assert int(host(out["error_flag"])[0]) == vsv.FLAG_LOGITS
        ids = host(out["ids"])
        assert np.all((ids >= 0) & (ids < V))
    y = x.clone()
    y[2] = -math.inf
    out = vsv.top_logits(y, 9)
    assert int(host(out["error_flag"])[0]) == vsv.FLAG_LOGITS
    assert np.array_equal(host(out["ids"])[2], np.arange(9))


# ------------------------------------------------------------- distillation

def _teacher(rng, xs, K, T, rest, repeat):
    n, V = len(xs), xs[0].shape[0]
    ids = np.full((n, K), -1, dtype=np.int32)
    z = np.full((n, K), np.nan, dtype=np.float32)
    lse = np.zeros(n, dtype=np.float32)
    for r, x in enumerate(xs):
        t = np.where(np.isfinite(x) & (x > -1e30), 0.6 * x, 0.0) + rng.standard_normal(V)
        used = min(K, V) if r % 4 else (min(K, V) + 1) // 2
        if r % 7 == 5:
            used = 0
        top = oracle.rank_order(t)[:used]
        if repeat and used > 2:
            top[2] = top[0]
        at = rng.permutation(K)[:used]                   # used entries anywhere
        ids[r, at], z[r, at] = top, t[top]
        lse[r] = oracle.logsumexp(t, T) + (0.3 if repeat else 0.0)
    return ids, z, (lse if rest else None)


def _check_distill(loss, grad, xs, ids, z, lse, T, w, dtype):
    for r, x in enumerate(xs):
        L = None if lse is None else float(lse[r])
        want, g = oracle.distill_row(x, ids[r], z[r].astype(np.float64), L, T, float(w[r]))
        if not np.any(ids[r] >= 0):
            assert loss[r] == 0 and (grad is None or not np.any(grad[r]))
            continue
        y = np.abs(x[ids[r][ids[r] >= 0]])      # named tokens count however far down they are
        D = 2.0 ** -22 * (1 + max(largest(x, T), y[np.isfinite(y)].max(initial=0.0) / T))
        want = float(np.float32(want)) if abs(want) > 1e38 else want
        if np.isfinite(want):
            assert abs(loss[r] - want) <= 2 * D + 2.0 ** -24 * abs(want), (r, loss[r], want)
        else:
            assert loss[r] == want, (r, loss[r], want)
        if grad is None:
            continue
        used = ids[r] >= 0
        q = np.exp(x / T - oracle.logsumexp(x, T))
        named = np.zeros(x.shape[0], dtype=bool)
        named[ids[r][used]] = True
        size = np.ones(x.shape[0])
        q_rest = q[~named].sum()
        if L is not None and q_rest > 0:
            t = np.exp(z[r][used].astype(np.float64) / T - L)
            size[~named] += max(0.0, 1 - t.sum()) / q_rest
        tol = 4 * D * q * size * w[r] / T + HALF[dtype] * np.abs(g) + 1e-37
        # the teacher's masses are rounded to float once
        tol[named] += 2.0 ** -23 * w[r] / T
        bad = np.flatnonzero(~(np.abs(grad[r] - g) <= tol))
        assert bad.size == 0, (r, bad[:5], grad[r][bad[:5]], g[bad[:5]], tol[bad[:5]])


def _f32(t):
    return host(t.float())


CASES = [(1, 1, 0, 0, 1.0), (7, 5, 1, 1, 2.0), (64, 64, 0, 0, 1.0), (1000, 17, 3, 1, 0.5), (4099, 256, 0, 3, 1.0),
         (20011, 64, 2, 0, 1.5)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rest", [False, True])
@pytest.mark.parametrize("V,K,pad,shift,T", CASES)
def test_distill(vsv, dtype, rest, V, K, pad, shift, T):
    n = 29
    kinds = ("plain", "ties", "masked", "equal", "spikes", "lowest")
    rng, x, xs = _store(60 + V, n, V, dtype, kinds, pad, shift)
    ids, z, lse = _teacher(rng, xs, K, T, rest, repeat=V > 100)
    w = rng.random(n, dtype=np.float32)
    w[4] = 0.0
    print("distill V=%d K=%d dtype=%d rest=%d" % (V, K, dtype, rest), flush=True)
    x = x[:, :V]
    args = (to_dev(ids), to_dev(z))
    kw = dict(teacher_lse=None if lse is None else to_dev(lse), temperature=T)
    loss, state = vsv.distill_forward(x, *args, **kw)
    grad = vsv.distill_backward(to_dev(w), x, *args, state, **kw)
    _check_distill(host(loss), _f32(grad), xs, ids, z, lse, T, w, dtype)
    loss2, grad2 = vsv.distill_loss_grad(x, *args, to_dev(w), **kw)
    _check_distill(host(loss2), _f32(grad2), xs, ids, z, lse, T, w, dtype)


@pytest.mark.parametrize("dtype,n", [(F32, 3), (BF16, 3), (F32, 530), (BF16, 530)])
def test_distill_over_a_full_vocabulary(vsv, dtype, n):
    # few rows are cut into parts, many are taken whole
    import torch
    V, K, T = 152064, 128, 1.0
    m = 3
    rng, x, xs = _store(77, m, V, dtype, ("plain", "spikes"), 0, 0)
    ids, z, lse = _teacher(rng, xs, K, T, True, True)
    w = rng.random(m, dtype=np.float32)
    pick = torch.arange(n, device="cuda") % m
    up = lambda a: to_dev(a)[pick].contiguous()
    loss, grad = vsv.distill_loss_grad(x[pick].contiguous(), up(ids), up(z), up(w), teacher_lse=up(lse))
    for r0 in (0, n - m) if n > m else (0,):
        order = host(pick[r0:r0 + m])
        _check_distill(host(loss)[r0:r0 + m], _f32(grad[r0:r0 + m]), [xs[q] for q in order], ids[order], z[order],
                       lse[order], T, w[order], dtype)
    # every copy of a row is the same row
    for q in range(m):
        same = grad[pick == q]
        assert bool((same == same[0]).all())


def test_distill_gradient_by_differences(vsv):
    # along a direction d: (loss(y + h d) - loss(y - h d)) / 2h against grad . d.
    # Losses are within 2 D (D as above, max|x| < 12): 2 D / h = 0.0031 at
    # h = 2^-7, and the third derivative of a log-sum-exp along |d| <= 1 is
    # below 1, so h^2 / 6 = 1e-5.
    import torch
    n, V, K, h = 12, 1003, 20, 2.0 ** -7
    rng, x, xs = _store(21, n, V, F32, ("plain",), 0, 0, sigma=1.0)
    ids, z, lse = _teacher(rng, xs, K, 1.0, True, True)
    d = torch.from_numpy(rng.uniform(-1, 1, (n, V)).astype(np.float32)).cuda()
    args = (to_dev(ids), to_dev(z), to_dev(lse))
    _, grad = vsv.distill_loss_grad(x, args[0], args[1], teacher_lse=args[2])
    up, dn = x + h * d, x - h * d
    diff = (vsv.distill_loss(up, *args).double() - vsv.distill_loss(dn, *args).double()) / (2 * h)
    along = (grad.double() * d.double()).sum(1)
    assert float(x.abs().max()) + h < 12
    tol = 2 * 2.0 ** -22 * (1 + 12) / h + h * h / 6
    assert float((diff - along).abs().max()) < tol


def test_distill_unused_and_foreign_entries(vsv):
    import torch
    V, n = 500, 6
    rng, x, xs = _store(31, n, V, BF16, ("plain",), 0, 0)
    x[1] = math.nan                              # a padding row holds anything
    ids = torch.tensor([[4, -1, 9]] * n, dtype=torch.int32, device="cuda")
    ids[1] = -5
    z = torch.tensor([[1.0, math.nan, 0.5]] * n, device="cuda")
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    loss, grad = vsv.distill_loss_grad(x, ids, z, error_flag=flag)
    assert float(loss[1]) == 0 and not bool(grad[1].any()) and int(flag) == 0
    assert bool(torch.isfinite(loss).all()) and bool(torch.isfinite(grad.float()).all())
    # an id at or beyond the vocabulary counts as unused and is flagged
    ids2 = ids.clone()
    ids2[3, 1] = V
    loss2, grad2 = vsv.distill_loss_grad(x, ids2, z, error_flag=flag)
    assert int(flag) == vsv.FLAG_TOKEN
    assert torch.equal(loss2, loss) and torch.equal(grad2, grad)
    # NaN in a row that counts
    flag.zero_()
    y = x.clone()
    y[2, 100] = math.nan
    vsv.distill_loss_grad(y, ids, z, error_flag=flag)
    assert int(flag) == vsv.FLAG_LOGITS
    # entries of weight 0 only name nothing
    loss3, grad3 = vsv.distill_loss_grad(x, ids, torch.full_like(z, -math.inf))
    assert not bool(loss3.any()) and not bool(grad3.any())


def test_student_that_excludes_the_teacher(vsv):
    # -inf at a teacher's token, or everywhere outside: an infinite loss, as
    # the formula says, and a finite gradient
    import torch
    x = torch.randn(2, 40, device="cuda")
    x[0, 3] = -math.inf
    x[1, 2:] = -math.inf
    ids = torch.tensor([[3, 5], [0, 1]], dtype=torch.int32, device="cuda")
    z = torch.zeros(2, 2, device="cuda")
    lse = torch.full((2,), 1.5, device="cuda")
    loss, grad = vsv.distill_loss_grad(x, ids, z, teacher_lse=lse)
    assert bool((loss == math.inf).all()) and bool(torch.isfinite(grad).all())
    w = np.ones(2)
    _check_distill(host(loss), host(grad), [host(q).astype(np.float64) for q in x], host(ids), host(z), host(lse), 1.0,
                   w, F32)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_distill_through_autograd(vsv, dtype):
    import torch
    n, V, K, width = 21, 999, 8, 1010
    rng, x, xs = _store(51, n, V, dtype, ("plain",), width - V, 0)
    ids, z, lse = _teacher(rng, xs, K, 1.3, True, False)
    args = (to_dev(ids), to_dev(z), to_dev(lse), 1.3)
    x = torch.where(torch.isnan(x), torch.zeros_like(x), x)
    leaf = x.clone().requires_grad_()
    loss = vsv.distill_loss(leaf * 1.0, *args, vocab=V)
    loss.sum().backward()                                  # one number for every row
    _check_distill(host(loss), _f32(leaf.grad)[:, :V], xs, ids, z, lse, 1.3, np.ones(n), dtype)
    assert not bool(leaf.grad[:, V:].any())                # columns that are no part of the rows
    w = torch.rand(n, device="cuda")
    g, = torch.autograd.grad(vsv.distill_loss(leaf, *args, vocab=V), leaf, w)
    _check_distill(host(loss), _f32(g)[:, :V], xs, ids, z, lse, 1.3, host(w), dtype)
    # a row broadcast to several: its gradient is their sum
    row = x[:1, :V].float().contiguous().requires_grad_()
    one = lambda t: t[:1].expand(5, *t.shape[1:]).contiguous()
    vsv.distill_loss(row.expand(5, V), *[one(t) for t in args[:3]], 1.3).sum().backward()
    _, g1 = oracle.distill_row(host(row)[0].astype(np.float64), ids[0], z[0].astype(np.float64), float(lse[0]), 1.3, 5.0)
    assert np.all(np.abs(host(row.grad)[0] - g1) <= 4 * 2.0 ** -22 * 20 * np.abs(g1) + 5 * 2.0 ** -22)


# ------------------------------------------------------- together, elsewhere

def test_draft_verify_and_learn(vsv):
    """One round as a server with a learning draft head runs it: drafts drawn
    from the head's rows, verified against the target's with the draft law,
    the target's top logits taken, and the head's rows graded against them."""
    import torch
    B, K, V = 24, 3, 4099
    rng = np.random.default_rng(90)
    target = torch.from_numpy(rng.standard_normal((B * (K + 1), V)).astype(np.float32) * 2).cuda()
    off = to_dev(np.arange(0, B * (K + 1) + 1, K + 1, dtype=np.int32))
    own = to_dev(np.repeat(np.arange(B, dtype=np.int32), K + 1))
    rows = torch.arange(B * (K + 1), device="cuda").view(B, K + 1)[:, :K].reshape(-1)
    head = (target[rows] * 0.8 + torch.randn(B * K, V, device="cuda") * 0.3).contiguous()
    n = B * K
    one, zero = torch.ones(n, device="cuda"), torch.zeros(n, device="cuda")
    u = torch.rand(n, device="cuda")
    drawn = vsv.sample_rows(head, one, torch.zeros(n, dtype=torch.int32, device="cuda"), one, zero, u)
    conf, _, _ = vsv.draft_confidence(head, drawn["token"])
    assert np.allclose(np.exp(host(drawn["logprob"])), host(conf), rtol=1e-5, atol=0)
    b1, b0 = torch.ones(B, device="cuda"), torch.zeros(B, device="cuda")
    out = vsv.verify_probabilistic(target, off, own, drawn["token"], head, b1,
                                   torch.zeros(B, dtype=torch.int32, device="cuda"), b1, b0, b1, seed=3)
    assert int(host(out["error_flag"])[0]) == 0
    acc = host(out["accepted_len"])
    assert acc.min() >= 0 and acc.max() <= K and acc.sum() > 0
    teacher = vsv.top_logits(target[rows].contiguous(), 32)
    leaf = head.requires_grad_()
    loss = vsv.distill_loss(leaf, teacher["ids"], teacher["values"], teacher["lse"])
    loss.mean().backward()
    w = np.full(n, np.float32(1) / np.float32(n))
    xs = [host(q).astype(np.float64) for q in head.detach()]
    _check_distill(host(loss), host(leaf.grad), xs, host(teacher["ids"]), host(teacher["values"]), host(teacher["lse"]),
                   1.0, w, F32)


def _calls(vsv, x, ids, z, lse, par):
    a = vsv.sample_rows(x, *par)
    b = vsv.top_logits(x, 33)
    loss, state = vsv.distill_forward(x, ids, z, lse)
    grad = vsv.distill_backward(par[0], x, ids, z, state, lse)
    loss2, grad2 = vsv.distill_loss_grad(x, ids, z, par[0], lse)
    return [a["token"], a["logprob"], a["lse"], b["values"], b["ids"], b["lse"], loss, grad, loss2, grad2]


def _together(n, V, dtype, seed):
    rng, x, xs = _store(seed, n, V, dtype, ("plain", "spikes"), 0, 0)
    ids, z, lse = _teacher(rng, xs, 30, 1.0, True, False)
    f = lambda v: to_dev(np.full(n, v, dtype=np.float32))
    par = (f(0.9), to_dev(np.full(n, 40, dtype=np.int32)), f(0.9), f(0.0), to_dev(rng.random(n, dtype=np.float32)))
    return x, to_dev(ids), to_dev(z), to_dev(lse), par


@pytest.mark.parametrize("n,V", [(5, 30000), (600, 1000)])
def test_calls_in_a_captured_graph(vsv, n, V):
    import torch
    args = _together(n, V, BF16, 71)
    other = _together(n, V, BF16, 72)
    want = [t.clone() for t in _calls(vsv, *args)]
    want2 = [t.clone() for t in _calls(vsv, *other)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        _calls(vsv, *args)
    torch.cuda.synchronize()
    x0 = args[0].clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        outs = _calls(vsv, *args)
    flat = lambda a: list(a[:4]) + list(a[4])
    keep = [t.clone() for t in flat(args)]
    for rep in range(4):
        src, ref = (keep, want) if rep % 2 == 0 else (flat(other), want2)
        for dst, t in zip(flat(args), src):
            dst.copy_(t)
        for o in outs:
            o.zero_()
        _calls(vsv, *other)                       # eager work between replays
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for i, (o, w) in enumerate(zip(outs, ref)):
            assert torch.equal(o, w), (rep, i)
    assert torch.equal(x0, keep[0])


def test_training_step_in_a_captured_graph(vsv):
    # forward and backward through autograd, on a leaf made for the capture
    import torch
    x, ids, z, lse, par = _together(40, 5000, F32, 73)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())

    def step():
        leaf = x.detach().requires_grad_()
        loss = vsv.distill_loss(leaf, ids, z, lse)
        return loss.detach(), torch.autograd.grad(loss, leaf, par[0])[0]

    with torch.cuda.stream(s):
        want = [t.clone() for t in step()]
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        outs = step()
    for _ in range(3):
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, w) for o, w in zip(outs, want))


def test_calls_on_two_streams_at_once(vsv):
    import torch
    cases = [_together(37, 20000, F32, 81), _together(37, 20000, F32, 82)]
    want = [[t.clone() for t in _calls(vsv, *c)] for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = [[], []]
    for _ in range(5):
        for i, (s, c) in enumerate(zip(streams, cases)):
            with torch.cuda.stream(s):
                got[i].append(_calls(vsv, *c))
    torch.cuda.synchronize()
    for i in range(2):
        for outs in got[i]:
            assert all(torch.equal(o, w) for o, w in zip(outs, want[i]))


def test_calls_given_a_stream(vsv):
    import torch
    x, ids, z, lse, par = _together(9, 20000, BF16, 83)
    want = [t.clone() for t in _calls(vsv, x, ids, z, lse, par)]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    a = vsv.sample_rows(x, *par, stream=s)
    b = vsv.top_logits(x, 33, stream=s)
    loss, state = vsv.distill_forward(x, ids, z, lse, stream=s)
    grad = vsv.distill_backward(par[0], x, ids, z, state, lse, stream=s)
    loss2, grad2 = vsv.distill_loss_grad(x, ids, z, par[0], lse, stream=s)
    s.synchronize()
    got = [a["token"], a["logprob"], a["lse"], b["values"], b["ids"], b["lse"], loss, grad, loss2, grad2]
    assert all(torch.equal(o, w) for o, w in zip(got, want))


def test_no_rows(vsv):
    import torch
    x = torch.empty(0, 50, device="cuda")
    f, i = torch.empty(0, device="cuda"), torch.empty(0, dtype=torch.int32, device="cuda")
    assert vsv.sample_rows(x, f, i, f, f, f)["token"].numel() == 0
    assert vsv.top_logits(x, 4)["ids"].shape == (0, 4)
    e = torch.empty(0, 3, device="cuda")
    loss, grad = vsv.distill_loss_grad(x, e.int(), e)
    assert loss.numel() == 0 and grad.shape == (0, 50)
    leaf = x.clone().requires_grad_()
    vsv.distill_loss(leaf, e.int(), e).sum().backward()
    assert leaf.grad.shape == (0, 50)


def test_neighbouring_memory_is_left_alone(vsv):
    # outputs in the middle of larger buffers, through the C entry points
    import ctypes
    import torch
    n, V, K, ld = 5, 1003, 12, 1010
    rng, x, xs = _store(61, n, V, F32, ("plain",), ld - V, 0)
    ids, z, lse = _teacher(rng, xs, K, 1.0, True, False)
    ids, z, lse = to_dev(ids), to_dev(z), to_dev(lse)
    L = vsv.lib()
    grad = torch.full((n + 2, ld), 77.0, device="cuda")
    loss = torch.full((n + 2,), 77.0, device="cuda")
    d = vsv.Distill(x.data_ptr(), 0, V, ld, n, K, ids.data_ptr(), z.data_ptr(), lse.data_ptr(), 1.0)
    need = L.vsv_distill_workspace_bytes(n, V, 0)
    ws = torch.full((need // 8 + 4,), 77.0, dtype=torch.float64, device="cuda")
    st = L.vsv_distill_grad(ctypes.byref(d), None, loss[1:].data_ptr(), grad[1:].data_ptr(), ld, None,
                            ws[1:].data_ptr(), need, torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert st == 0
    _check_distill(host(loss)[1:-1], host(grad)[1:-1, :V], xs, host(ids), host(z), host(lse), 1.0, np.ones(n), F32)
    assert bool((grad[1:-1, V:] == 77).all()) and bool((grad[0] == 77).all()) and bool((grad[-1] == 77).all())
    assert float(loss[0]) == 77 and float(loss[-1]) == 77
    assert float(ws[0]) == 77 and bool((ws[need // 8 + 1:] == 77).all())
