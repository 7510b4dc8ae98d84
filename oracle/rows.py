"""Plain float64 definitions of the logit-row operators next to verification:
one drawn token per row, a teacher's top logits, distillation.

One row at a time, written from the formulas; the draw itself is
oracle.verify's filtered_support. Test infrastructure only.
"""
import math

import numpy as np

from .verify import filtered_support, greedy_token, logsumexp, rank_order


def draw_row(x, temperature, top_k, top_p, min_p, u):
    """(token, log-probability under the filtered law, log-sum-exp of x / T)
    of one row; temperature 0 takes the arg-max."""
    if temperature == 0.0:
        return greedy_token(x), 0.0, logsumexp(x)
    S, w = filtered_support(x, temperature, top_k, top_p, min_p)
    c = np.cumsum(w[S])
    t = int(S[int(np.flatnonzero(c > u * c[-1])[0])])
    return t, float((x[t] - np.max(x)) / temperature - math.log(c[-1])), logsumexp(x, temperature)


def top_row(x, k, temperature=1.0):
    """(values, tokens) of the k first tokens in rank order and the row's
    log-sum-exp of x / temperature."""
    ids = rank_order(x)[:k]
    return x[ids], ids, logsumexp(x, temperature)


def distill_row(y, ids, z, teacher_lse, temperature, weight=1.0):
    """(loss, weight * gradient in y) of one student row against entries
    (ids, z); negative ids are unused, teacher_lse None renormalises the
    teacher over its entries. A rest of the teacher within the rounding of a
    float32 teacher_lse counts as none where the student's is below 2^-126."""
    ids, z = np.asarray(ids), np.asarray(z, dtype=np.float64)
    used = ids >= 0
    grad = np.zeros(y.shape[0])
    ids, z = ids[used], z[used] / temperature
    if ids.size == 0 or (teacher_lse is None and np.all(np.isneginf(z))):
        return 0.0, grad
    t = np.exp(z - (logsumexp(z) if teacher_lse is None else teacher_lse))
    log_q = y / temperature - logsumexp(y, temperature)
    q = np.exp(log_q)
    on = t > 0
    with np.errstate(divide="ignore"):
        loss = float(np.sum(t[on] * (np.log(t[on]) - log_q[ids[on]])))
        named = np.zeros(y.shape[0], dtype=bool)
        named[ids] = True
        rest = 0.0 if teacher_lse is None else max(0.0, 1.0 - float(np.sum(t)))
        # (by logarithms: q_rest may lie far below the smallest float64)
        log_rest = logsumexp(y[~named], temperature) if np.any(y[~named] > -np.inf) else -np.inf
        log_q_rest = log_rest - logsumexp(y, temperature)
        if log_q_rest < -126 * math.log(2) and rest <= 2.0 ** -20 * (1 + abs(teacher_lse or 0.0)):
            rest = 0.0                           # the rounding of a float32 teacher_lse
        total = float(np.sum(t)) + rest
        grad = q * total
        if rest > 0.0:
            loss += rest * (math.log(rest) - log_q_rest)
            if log_rest > -np.inf:
                grad[~named] -= rest * np.exp(y[~named] / temperature - log_rest)
    np.subtract.at(grad, ids, t)
    return loss, weight * grad / temperature
