"""Trees of drafts over a paged cache: CPU oracle (float64 NumPy, test
infrastructure only).

A request's packed rows are the nodes of a tree: its first row is the root
(the last token already emitted), every later row a draft whose parent is an
earlier row of the request; a chain is the tree whose row j hangs on row
j - 1. The pages name tree verification as a mode of the EAGLE path without
its rules (vllm-hust-vspec 0.13.0 README, "Scope of support"). Readings
taken: acceptance is strict, the walk takes the lowest fitting row, a row's
attention and penalties see its own path alone.

Pinned by tests/test_oracle_tree.py: chains against the linear oracle, closed
forms, brute force over tiny trees.
"""
import numpy as np

from .verify import bf16_bits_to_f64, greedy_token, logsumexp, row_f64


def path_of(parents, j):
    """Rows of a request from its root to row j; parents None: a chain."""
    path = [j]
    while path[0] > 0:
        path.insert(0, path[0] - 1 if parents is None else int(parents[path[0]]))
    return path


def verify_greedy_tree(logits, dtype, vocab, offsets, drafts, parents=None):
    """Greedy verification of trees; rows of a path root first in out_rows."""
    off = [int(o) for o in offsets]
    B, R = len(off) - 1, off[-1]
    token = [greedy_token(row_f64(logits, dtype, r, vocab)) for r in range(R)]
    lse = [logsumexp(row_f64(logits, dtype, r, vocab)) for r in range(R)]
    acc, nxt, out_off, toks, rows = [], [], [0], [], []
    for i in range(B):
        r0, r1 = off[i], off[i + 1]
        at, path = r0, [r0]
        while True:
            for r in range(at + 1, r1):
                up = r - r0 - 1 if parents is None else int(parents[r])
                if r0 + up == at and int(drafts[r - i - 1]) == token[at]:
                    break
            else:
                break
            toks.append(token[at])
            at = r
            path.append(r)
        acc.append(len(path) - 1)
        nxt.append(token[at])
        toks.append(token[at])
        rows += path
        out_off.append(len(rows))
    i32 = lambda a: np.array(a, dtype=np.int32)
    return dict(accepted_len=i32(acc), next_token=i32(nxt), out_offsets=i32(out_off), out_tokens=i32(toks),
                out_rows=i32(rows), row_token=i32(token), row_lse=np.array(lse))


def adjust_row(x, prompt, output, repetition=1.0, frequency=0.0, presence=0.0, bias=(), allowed=None):
    """One row after penalties, biases and mask. `prompt` and `output` (drafts
    of the row's path among them) are lists of tokens, `bias` pairs of token
    and value (the last of a token counts), `allowed` truth values [V]."""
    y = np.array(x, dtype=np.float64)
    count = np.bincount(np.asarray(output, dtype=np.int64), minlength=y.size)
    seen = count + np.bincount(np.asarray(prompt, dtype=np.int64), minlength=y.size) > 0
    y[seen] = np.where(y[seen] > 0, y[seen] / repetition, y[seen] * repetition)
    y[count > 0] -= frequency * count[count > 0] + presence
    for t, v in dict(bias).items():
        y[t] += v
    if allowed is not None:
        y[~np.asarray(allowed, dtype=bool)] = -np.inf
    return y


def plan_pages(table, held, length, offsets, free_pages, free_count, page_size, num_rows):
    """Page plan on copies; see vsv_plan_pages. Returns a dict, with
    `short` true if the pool ran out."""
    table, pool = np.array(table), np.array(free_pages)
    held, length = np.array(held), np.array(length)
    off = [int(o) for o in offsets]
    B, top = len(off) - 1, int(free_count)
    rows = [off[i + 1] - off[i] for i in range(B)]
    need = [-(-(int(length[i]) + rows[i]) // page_size) for i in range(B)]
    for i in range(B):
        for p in range(need[i], int(held[i])):
            pool[top] = table[i, p]
            top += 1
    slot = np.full(num_rows, -1, dtype=np.int64)
    position = np.full(num_rows, -1, dtype=np.int32)
    short = False
    for i in range(B):
        take = need[i] - int(held[i])
        if take > 0 and (short or take > top):
            short = True
            continue
        for p in range(int(held[i]), need[i]):
            top -= 1
            table[i, p] = pool[top]
        held[i] = need[i]
        for j in range(rows[i]):
            at = int(length[i]) + j
            position[off[i] + j] = at
            slot[off[i] + j] = int(table[i, at // page_size]) * page_size + at % page_size
        length[i] += rows[i]
    return dict(slot=slot, position=position, held=held, length=length, free_count=np.array([top], dtype=np.int32),
                block_table=table, free_pages=pool, short=short)


def _f64(a):
    a = np.asarray(a)
    return bf16_bits_to_f64(a) if a.dtype == np.uint16 else a.astype(np.float64)


def tree_attention(q, k, v, offsets, k_cache, v_cache, table, length, parents=None, scale=None):
    """Attention of every row over its request's cached tokens, its own path
    and itself; q [R, H, D], k and v [R, KV, D], caches [pages, page, KV, D]
    (float32, or uint16 bfloat16 bits). Returns (out, lse) in float64."""
    q, k, v, kc, vc = [_f64(a) for a in (q, k, v, k_cache, v_cache)]
    R, H, D = q.shape
    KV, page = k.shape[1], kc.shape[1]
    scale = D ** -0.5 if scale is None else scale
    out, lse = np.zeros((R, H, D)), np.zeros((R, H))
    for i in range(len(offsets) - 1):
        r0, r1, n = int(offsets[i]), int(offsets[i + 1]), int(length[i])
        ids = [int(table[i, t // page]) for t in range(n)]
        at = [t % page for t in range(n)]
        for r in range(r0, r1):
            own = [r0 + j for j in path_of(None if parents is None else parents[r0:r1], r - r0)]
            for h in range(H):
                g = h // (H // KV)
                keys = np.concatenate((kc[ids, at, g].reshape(-1, D), k[own, g]))
                vals = np.concatenate((vc[ids, at, g].reshape(-1, D), v[own, g]))
                s = keys @ q[r, h] * scale
                m = s.max()
                w = np.exp(s - m)
                lse[r, h] = m + np.log(w.sum())
                out[r, h] = w @ vals / w.sum()
    return out, lse
