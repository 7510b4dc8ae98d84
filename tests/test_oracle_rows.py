"""Pins of the row operators' oracle: closed forms, brute force, differences."""
import math

import numpy as np
import pytest

import oracle


def test_draw_on_a_law_written_down():
    # weights 8 : 4 : 2 : 2 at T = 1, tokens 2, 0, 1, 3 in rank order
    x = np.log(np.array([4.0, 2.0, 8.0, 2.0]))
    for u, t in ((0.0, 2), (0.499, 2), (0.501, 0), (0.749, 0), (0.751, 1), (0.874, 1), (0.876, 3), (0.999, 3)):
        tok, lp, lse = oracle.draw_row(x, 1.0, 0, 1.0, 0.0, u)
        assert tok == t
        assert math.isclose(lp, math.log(math.exp(x[t]) / 16.0), rel_tol=1e-12)
        assert math.isclose(lse, math.log(16.0), rel_tol=1e-12)
    # top-k 2 leaves 8 : 4; top-p 0.6 of those leaves the first alone
    assert oracle.draw_row(x, 1.0, 2, 1.0, 0.0, 0.7)[0] == 0
    assert math.isclose(oracle.draw_row(x, 1.0, 2, 1.0, 0.0, 0.7)[1], math.log(1 / 3), rel_tol=1e-12)
    assert oracle.draw_row(x, 1.0, 2, 0.6, 0.0, 0.99)[:2] == (2, 0.0)
    # min-p 0.4 leaves 8 : 4
    assert oracle.draw_row(x, 1.0, 0, 1.0, 0.4, 0.99)[0] == 0
    assert oracle.draw_row(x, 0.0, 0, 1.0, 0.0, 0.9)[:2] == (2, 0.0)


def test_draw_frequencies_are_the_law():
    x = np.array([0.3, -1.0, 2.0, 0.3, -np.inf])
    n = 4096
    got = np.bincount([oracle.draw_row(x, 0.8, 0, 1.0, 0.0, (i + 0.5) / n)[0] for i in range(n)], minlength=5) / n
    p = np.exp(x / 0.8) / np.sum(np.exp(x / 0.8))
    assert np.all(np.abs(got - p) <= 2.0 / n)


def test_top_rows_break_ties_by_index():
    v, ids, lse = oracle.top_row(np.array([1.0, 3.0, -0.0, 3.0, 0.0]), 4)
    assert ids.tolist() == [1, 3, 0, 2] and v.tolist() == [3.0, 3.0, 1.0, 0.0]
    assert math.isclose(lse, math.log(math.exp(1) + 2 * math.exp(3) + 2), rel_tol=1e-12)


def test_distill_closed_forms():
    y = np.log(np.array([1.0, 2.0, 5.0]))
    # teacher equal to the student over the whole row: nothing to learn
    loss, g = oracle.distill_row(y, [2, 1, 0], y[[2, 1, 0]], oracle.logsumexp(y), 1.0)
    assert abs(loss) < 1e-14 and np.all(np.abs(g) < 1e-14)
    # one entry: cross-entropy
    loss, g = oracle.distill_row(y, [1, -1], [7.0, 9.0], None, 1.0)
    assert math.isclose(loss, math.log(4.0), rel_tol=1e-12)
    assert np.allclose(g, [0.125, 0.25 - 1.0, 0.625], rtol=0, atol=1e-15)
    # one entry of a quarter against the rest: a two-cell divergence
    loss, g = oracle.distill_row(y, [1], [math.log(0.25)], 0.0, 1.0)
    assert abs(loss) < 1e-14 and np.all(np.abs(g) < 1e-15)
    assert oracle.distill_row(y, [-1, -1], [1.0, 2.0], None, 1.0)[0] == 0.0


@pytest.mark.parametrize("rest", [False, True])
@pytest.mark.parametrize("repeat", [False, True])
def test_distill_gradient_by_differences(rest, repeat):
    rng = np.random.default_rng(4 + rest)
    y, T = rng.standard_normal(9) * 2, 1.7
    ids = np.array([3, 8, 3 if repeat else 0, -1])
    z = rng.standard_normal(4)
    lse = float(np.log(np.sum(np.exp(z[:3] / T))) + 0.6) if rest else None
    _, g = oracle.distill_row(y, ids, z, lse, T, 0.5)
    for i in range(9):
        h = 1e-5
        up, dn = y.copy(), y.copy()
        up[i] += h
        dn[i] -= h
        d = 0.5 * (oracle.distill_row(up, ids, z, lse, T)[0] - oracle.distill_row(dn, ids, z, lse, T)[0]) / (2 * h)
        assert abs(d - g[i]) < 1e-9      # h^2 of a smooth function of order 1, and 1e-16 / h


def test_distill_rest_that_is_a_rounding():
    # a mask that leaves only named tokens, on both sides: the float32
    # log-sum-exp leaves a rest of 1e-7, which is no mass without a student
    z = np.array([1.0, 0.25, -0.5])
    y = np.concatenate((z, np.full(5, -np.inf)))
    for mask in (-np.inf, float(np.finfo(np.float32).min)):
        y[3:] = mask
        loss, g = oracle.distill_row(y, [0, 1, 2], z, oracle.logsumexp(z) + 1e-7, 1.0)
        assert abs(loss) < 2e-7 and np.all(np.abs(g) < 2e-7)
    # a rest that is more than that stays: against nothing it is infinite
    assert oracle.distill_row(y, [0, 1], z[:2], oracle.logsumexp(z), 1.0)[0] < 10.0     # token 2 is outside
    y[3:] = -np.inf
    assert oracle.distill_row(y, [0, 1, 2], z, oracle.logsumexp(z) + 1e-3, 1.0)[0] == np.inf
    # and one within it counts where the student has a rest
    y[3:] = -20.0
    loss, _ = oracle.distill_row(y, [0, 1, 2], z, oracle.logsumexp(z) + 1e-7, 1.0)
    q = 5 * math.exp(-20.0 - oracle.logsumexp(y))
    want = -1e-7 - math.log1p(-q) + 1e-7 * (math.log(1e-7) - math.log(q))
    assert abs(loss - want) < 1e-12
