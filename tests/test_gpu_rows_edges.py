"""The row operators at the edges of what they accept, against the float64
definition. Tolerances are those derived in test_gpu_rows.py unless a test
states its own."""
import math

import numpy as np
import pytest

import oracle
from tests.row_cases import BF16, F32, rows_f64, store_rows
from tests.test_gpu_rows import _check_draws
from tests.workloads import cuda_or_skip, host, to_dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def vsv():
    cuda_or_skip()
    import draft_token_verification_packed_amd as m
    m.lib()
    return m


# ------------------------------------------------------------------- draws

@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("V", [300, 70001])
def test_draws_at_subnormal_temperatures(vsv, dtype, V):
    # bins narrower than the smallest float: only the row's largest elements
    # hold weight, or its subnormal ones where the type has any below T
    rng = np.random.default_rng(2)
    rows = []
    for kind in range(4):
        x = np.zeros(V, dtype=np.float32)
        if kind == 1:
            x[rng.random(V) < 0.7] = -1.0
        elif kind == 2:
            x[rng.random(V) < 0.7] = -0.0
        elif kind == 3:
            x -= (rng.integers(0, 40, V) * 2.0 ** -149).astype(np.float32)
        rows.append(x)
    T = np.array([1.4e-45, 1e-44, 8e-44, 1e-43, 1e-42, 1e-40], dtype=np.float32)
    n = len(rows) * len(T)
    store = store_rows([rows[r % 4] for r in range(n)], dtype)
    a = (np.repeat(T, 4), np.full(n, 0, dtype=np.int32), np.where(np.arange(n) % 2, 0.9, 1.0).astype(np.float32),
         np.where(np.arange(n) % 3, 0.0, 0.05).astype(np.float32), rng.random(n, dtype=np.float32))
    print("subnormal temperatures V=%d dtype=%d" % (V, dtype), flush=True)
    _check_draws(vsv.sample_rows(to_dev(store), *[to_dev(q) for q in a]), rows_f64(store, dtype, V, 0), *a)


def _tied_bulk(bulk, z):
    """(weight of a bulk token, total) of a row with one token at 0, `bulk` at
    -z and the others at -inf, in 64-bit mantissas."""
    w = np.exp(-np.longdouble(z))
    return w, 1 + bulk * w


def _rounded(V, bulk, z):
    """The same with weights rounded to 2^-s, s the most that V of them allow
    in 62 bits."""
    s = min(50, 62 - int(V).bit_length())
    w = np.rint(np.exp(-np.longdouble(z)) * 2.0 ** s) / np.longdouble(2.0 ** s)
    return w, 1 + bulk * w


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("V,bulk,z", [(152064, 4000, 18.0), (20000, 19999, 17.0), (70001, 70000, 16.0), (152064, 152063, 12.0), (152064, 152063, 15.0)])
def test_draws_among_many_equal_tokens_far_below_the_maximum(vsv, dtype, V, bulk, z):
    # thousands of equal weights round alike, so weights rounded relative to
    # the row's maximum add up to a neighbouring token towards the end. The
    # numbers are those where that shows, at least 1e-4 of a token's share
    # off its borders (sums within 1e-13 of the total are 7e-6 of a share).
    w, total = _tied_bulk(bulk, z)
    wr, totalr = _rounded(V, bulk, z)
    first = int(2 ** 24 / total) + 1
    u = np.arange(first, 2 ** 24).astype(np.longdouble) / 2 ** 24
    at = (u * total - 1) / w
    off = (u * totalr - 1) / wr
    inside = np.abs(at - np.rint(at)) > 1e-4
    wrong = np.flatnonzero((np.floor(at) != np.floor(off)) & inside)
    right = np.flatnonzero((np.floor(at) == np.floor(off)) & inside)
    rng = np.random.default_rng(12)
    assert wrong.size >= 3
    pick = np.concatenate((rng.choice(wrong, min(20, wrong.size), replace=False), rng.choice(right, 4)))
    n = pick.size
    row = np.full(V, -np.inf, dtype=np.float32)
    lead = bulk // 3
    row[:bulk + 1] = -z
    row[lead] = 0.0
    par = [np.full(n, v, dtype=t) for v, t in ((1.0, np.float32), (0, np.int32), (1.0, np.float32), (0.0, np.float32))]
    print("many equal tokens V=%d bulk=%d z=%g dtype=%d" % (V, bulk, z, dtype), flush=True)
    out = vsv.sample_rows(to_dev(store_rows([row] * n, dtype)), *[to_dev(q) for q in par],
                          to_dev(u[pick].astype(np.float32)))
    rank = np.floor(at[pick]).astype(np.int64)
    assert np.array_equal(host(out["token"]), rank + (rank >= lead))
    want = float(-z - np.log(total))
    assert np.all(np.abs(host(out["logprob"]) - want) <= 2.0 ** -24 * abs(want) + 1e-9)
    assert np.all(np.abs(host(out["lse"]) - float(np.log(total))) <= 2.0 ** -24 * float(np.log(total)) + 1e-9)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_top_p_among_many_equal_tokens_far_below_the_maximum(vsv, dtype):
    # where the cut falls shows in the leading token's log-probability: a
    # token more or less is 3e-7 of it, its rounding 3e-9
    V, z = 152064, 15.0
    w, total = _tied_bulk(V - 1, z)
    wr, totalr = _rounded(V, V - 1, z)
    p = np.arange(int(2 ** 24 / total) + 1, 2 ** 24).astype(np.longdouble) / 2 ** 24
    need = (p * total - 1) / w                   # bulk tokens that reach it
    off = (p * totalr - 1) / wr
    wrong = np.flatnonzero((np.ceil(need) != np.ceil(off)) & (np.abs(need - np.rint(need)) > 1e-5))
    pick = np.random.default_rng(13).choice(wrong, 24, replace=False)
    n = pick.size
    row = np.full(V, -z, dtype=np.float32)
    row[7] = 0.0
    full = lambda v, t: to_dev(np.full(n, v, dtype=t))
    out = vsv.sample_rows(to_dev(store_rows([row] * n, dtype)), full(1.0, np.float32), full(0, np.int32),
                          to_dev(p[pick].astype(np.float32)), full(0.0, np.float32), full(0.0, np.float32))
    assert np.all(host(out["token"]) == 7)
    want = -np.log(1 + np.ceil(need[pick]) * w).astype(np.float64)
    assert np.all(np.abs(host(out["logprob"]) - want) <= 2.0 ** -24 * np.abs(want) + 1e-9)


@pytest.mark.parametrize("V", [152064, 70001])
@pytest.mark.parametrize("rise", [24.1, 24.6, 25.2, 40.0])
def test_draws_of_a_bulk_far_below_another_parts_maximum(vsv, V, rise):
    # every part of the row but the last holds a flat bulk, the last one token
    # `rise` above its middle: the bulk still weighs 4e-6 of it at 24.1, and
    # numbers close to one draw from it. A bulk token's share is down to 4e-12
    # there, so sums within 1e-13 of the total tell the tokens apart where a
    # number lies a tenth of a share off the borders.
    rng = np.random.default_rng(31)
    n = 12
    bulk = V * 7 // 8 if V > 100000 else V // 2
    rows, want, us = [], [], []
    for r in range(n):
        x = np.full(V, -np.inf, dtype=np.float32)
        x[:bulk] = rng.uniform(-1, 1, bulk)
        x[V - 1 - r] = np.float32(rise)
        ids = oracle.rank_order(x.astype(np.float64))[:bulk + 1]
        xl = x.astype(np.longdouble)
        w = np.exp(xl[ids] - xl[ids[0]])
        c = np.cumsum(w)
        token, u = V - 1 - r, 0.5
        if r % 4:
            for i in range(1, 80):
                t = (1 - np.longdouble(i) / 2 ** 24) * c[-1]
                k = int(np.searchsorted(c, t, side="right"))
                if k > 0 and min(t - c[k - 1], c[k] - t) > 0.1 * w[k] and i % 4 == r % 4:
                    token, u = int(ids[k]), 1 - i * 2.0 ** -24
                    break
        rows.append(x)
        us.append(u)
        want.append((token, float(xl[token] - xl[ids[0]] - np.log(c[-1])), float(xl[ids[0]] + np.log(c[-1]))))
    assert rise > 30 or sum(u > 0.6 for u in us) >= 6
    full = lambda v, t: to_dev(np.full(n, v, dtype=t))
    out = vsv.sample_rows(to_dev(store_rows(rows, F32)), full(1.0, np.float32), full(0, np.int32), full(1.0, np.float32),
                          full(0.0, np.float32), to_dev(np.array(us, dtype=np.float32)))
    tok, lp, lse = host(out["token"]), host(out["logprob"]), host(out["lse"])
    for r, (t, p, s) in enumerate(want):
        assert int(tok[r]) == t, (r, us[r], int(tok[r]), t)
        assert abs(lp[r] - p) <= 2.0 ** -24 * abs(p) + 1e-9, (r, lp[r], p)
        assert abs(lse[r] - s) <= 2.0 ** -24 * abs(s) + 1e-9, (r, lse[r], s)


# ------------------------------------------------------------- distillation

def _both(vsv, x, ids, z, w, **kw):
    """(loss, gradient) in one call, and by the two halves."""
    loss, state = vsv.distill_forward(x, ids, z, **kw)
    return vsv.distill_loss_grad(x, ids, z, w, **kw), (loss, vsv.distill_backward(w, x, ids, z, state, **kw))


def _check_rest(loss, grad, xs, ids, z, lse, T, w, dtype):
    """As _check_distill of test_gpu_rows.py, for rows whose mass outside the
    ids may be too small for a float64. With s the softmax over the unnamed
    tokens alone, their gradient is (M q - t_r s) weight / T, and both terms
    are exponentials within D, so it is within 4 D (M q + t_r s) weight / T;
    D counts the largest |x| / T of every token, named or not."""
    half = {F32: 2.0 ** -24, BF16: 2.0 ** -8}[dtype]
    for r, x in enumerate(xs):
        want, g = oracle.distill_row(x, ids[r], z[r].astype(np.float64), float(lse[r]), T, float(w[r]))
        D = 2.0 ** -22 * (1 + np.abs(x[np.isfinite(x)]).max() / T)
        if np.isfinite(want):
            assert abs(loss[r] - want) <= 2 * D + 2.0 ** -24 * abs(want), (r, loss[r], want)
        else:
            assert loss[r] == want, (r, loss[r], want)
        named = np.zeros(x.shape[0], dtype=bool)
        named[ids[r][ids[r] >= 0]] = True
        size = np.exp(x / T - oracle.logsumexp(x, T))
        rest = x[~named]
        if np.any(rest > -np.inf):
            t_r = max(0.0, 1 - np.exp(z[r][ids[r] >= 0].astype(np.float64) / T - float(lse[r])).sum())
            size[~named] += t_r * np.exp(rest / T - oracle.logsumexp(rest, T))
        tol = (4 * D * size + 2.0 ** -23 * named) * w[r] / T + half * np.abs(g) + 1e-37
        bad = np.flatnonzero(~(np.abs(grad[r] - g) <= tol))
        assert bad.size == 0, (r, bad[:5], grad[r][bad[:5]], g[bad[:5]], tol[bad[:5]])


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("V,n", [(4099, 5), (152064, 5), (152064, 130)])
@pytest.mark.parametrize("T", [0.5, 1.0])
def test_distill_of_a_student_far_above_the_rest(vsv, dtype, V, n, T):
    # the named logits lie so far above the others that the mass outside them
    # leaves the range of a float, then of a double: loss and gradient are
    # finite all the same. Rows in one workgroup and in parts.
    import torch
    gaps, K = (60, 90, 200, 700, 3000), 12
    m = len(gaps)
    rng = np.random.default_rng(44)
    ids = np.stack([rng.permutation(V)[:K] for _ in range(m)]).astype(np.int32)
    ids[:, 3] = ids[:, 0]                         # (named twice)
    rows = []
    for r, gap in enumerate(gaps):
        x = rng.standard_normal(V).astype(np.float32)
        x[ids[r]] += np.float32(gap * T)
        rows.append(x)
    z = rng.standard_normal((m, K)).astype(np.float32)
    lse = np.array([oracle.logsumexp(q.astype(np.float64), T) + 0.1 for q in z], dtype=np.float32)
    w = rng.random(m, dtype=np.float32)
    store = store_rows(rows, dtype)
    xs = rows_f64(store, dtype, V, 0)
    pick = torch.arange(n, device="cuda") % m
    up = lambda a: to_dev(a)[pick].contiguous()
    print("far above the rest V=%d n=%d dtype=%d" % (V, n, dtype), flush=True)
    for loss, grad in _both(vsv, up(store), up(ids), up(z), up(w), teacher_lse=up(lse), temperature=T):
        _check_rest(host(loss)[:m], host(grad[:m].float()), xs, ids, z, lse, T, w, dtype)
        assert bool((grad == grad[:m][pick]).all()) and bool((loss == loss[:m][pick]).all())


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("mask", ["inf", "lowest"])
@pytest.mark.parametrize("V,left,K,T", [(64, 64, 64, 1.0), (4099, 50, 64, 1.0), (4099, 256, 256, 0.7), (4099, 1, 8, 1.0),
                                        (152064, 90, 100, 2.0)])
def test_distill_on_a_masked_vocabulary(vsv, dtype, mask, V, left, K, T):
    # top_logits into distill_loss where a mask leaves at most K tokens, on
    # both sides: what float32 leaves of one is no mass to hold against the
    # student, so a student like the teacher has next to no loss
    from tests.row_cases import LOWEST
    rng = np.random.default_rng(V + left)
    n = 16
    rows = []
    for r in range(n):
        x = np.full(V, -np.inf if mask == "inf" else LOWEST[dtype], dtype=np.float32)
        x[rng.permutation(V)[:left]] = rng.standard_normal(left) * 3 + rng.uniform(-30, 30)
        rows.append(x)
    store = store_rows(rows, dtype)
    x, xs = to_dev(store), rows_f64(store, dtype, V, 0)
    top = vsv.top_logits(x, K, temperature=T)
    args = (x, top["ids"], top["values"])
    w = np.ones(n, dtype=np.float32)
    print("masked V=%d left=%d dtype=%d" % (V, left, dtype), flush=True)
    ids, z, lse = host(top["ids"]), host(top["values"]), host(top["lse"])
    for loss, grad in _both(vsv, *args, to_dev(w), teacher_lse=top["lse"], temperature=T):
        loss, grad = host(loss), host(grad.float())
        for r in range(n):
            want, g = oracle.distill_row(xs[r], ids[r], z[r].astype(np.float64), float(lse[r]), T)
            # logits that hold weight lie within 43 of zero; the teacher's
            # log-sum-exp is off by D too
            D = 2.0 ** -22 * (1 + 43 / T)
            assert abs(want) <= 3 * D and abs(loss[r] - want) <= 2 * D, (r, loss[r], want)
            assert np.all(np.abs(grad[r] - g) <= 4 * D / T + 2.0 ** -8 * np.abs(g)), r
            assert np.all(np.abs(grad[r]) <= 8 * D / T), r


def test_distill_refuses_forward_mode(vsv):
    import torch
    import torch.autograd.forward_ad as fw
    x = torch.randn(3, 50, device="cuda")
    ids = torch.tensor([[1, 4]] * 3, dtype=torch.int32, device="cuda")
    z = torch.zeros(3, 2, device="cuda")
    want = vsv.distill_loss(x, ids, z)
    with fw.dual_level():
        with pytest.raises(NotImplementedError):
            vsv.distill_loss(fw.make_dual(x, torch.ones_like(x)), ids, z)
        assert torch.equal(vsv.distill_loss(x, ids, z), want)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_rows_without_entries_are_not_read_in_parts(vsv, dtype):
    # few long rows are summed in parts, which leave their sums in the
    # scratch: nothing is left for a row without a used entry
    import ctypes
    import torch
    n, V, K = 5, 152064, 6
    x = torch.randn(n, V, device="cuda").to(torch.bfloat16 if dtype == BF16 else torch.float32)
    ids = torch.randint(0, V, (n, K), dtype=torch.int32, device="cuda")
    ids[1], ids[4], ids[2, 1:] = -1, -7, -1
    z, lse = torch.randn(n, K, device="cuda"), torch.full((n,), 3.0, device="cuda")
    L = vsv.lib()
    need = L.vsv_distill_workspace_bytes(n, V, dtype)
    assert need > 0
    for teacher_lse in (None, lse):
        ws = torch.full((need // 8,), 77.0, dtype=torch.float64, device="cuda")
        loss = torch.full((n,), 77.0, device="cuda")
        d = vsv.Distill(x.data_ptr(), dtype, V, V, n, K, ids.data_ptr(), z.data_ptr(),
                        None if teacher_lse is None else lse.data_ptr(), 1.0)
        assert L.vsv_distill_forward(ctypes.byref(d), loss.data_ptr(), None, None, ws.data_ptr(), need,
                                     torch.cuda.current_stream().cuda_stream) == 0
        per = (need // 8 - n * vsv.DISTILL_STATE) // n
        left = host((ws[:n * per].view(n, per) == 77).all(1))
        assert left.tolist() == [False, True, False, False, True]
        assert torch.equal(loss, vsv.distill_loss(x, ids, z, teacher_lse))
        assert float(loss[1]) == 0 and float(loss[4]) == 0 and bool((loss[[0, 2, 3]] != 77).all())
