"""Cases of the operators of one verification round over a paged cache.

`run` computes each operator in its plain form, or (own = True) through the
framework's entry points:
    tree_attention      attention of packed draft rows (chains or trees) over
                        a paged cache and the rows' own keys and values
    adjust_logits       penalties, biases and grammar masks on packed rows
    verify_greedy_tree  greedy acceptance along a path of a tree of drafts
    plan_pages          block tables and slots from lengths on the device
"""
import math

import torch

own = False

VOCAB = 152064


def listed():
    return [
        # one request's verify rows, a chain of four drafts: what a single
        # user waits for
        dict(name="attn_step_bf16", op="attn", dtype="bf16", requests=1, rows_lo=5, rows_hi=5, len_lo=1024, len_hi=1024,
             heads=40, kv_heads=8, dim=128, page=16, tree="chain"),
        # a full serving batch of the same chains
        dict(name="attn_verify_bf16", op="attn", dtype="bf16", requests=128, rows_lo=5, rows_hi=5, len_lo=200,
             len_hi=1019, heads=40, kv_heads=8, dim=128, page=16, tree="chain"),
        # trees of up to 50 nodes: the compute-heavy end
        dict(name="attn_tree_bf16", op="attn", dtype="bf16", requests=16, rows_lo=20, rows_hi=50, len_lo=1000,
             len_hi=8000, heads=40, kv_heads=8, dim=128, page=32, tree="wide"),
        # two long documents
        dict(name="attn_long_bf16", op="attn", dtype="bf16", requests=2, rows_lo=3, rows_hi=8, len_lo=49153,
             len_hi=65000, heads=64, kv_heads=8, dim=128, page=64, tree="wide"),
        # a small draft model in fp32: odd group, empty contexts among the requests
        dict(name="attn_odd_f32", op="attn", dtype="f32", requests=9, rows_lo=1, rows_hi=17, len_lo=0, len_hi=1001,
             heads=14, kv_heads=2, dim=64, page=16, tree="wide"),
        # the smallest call: a toy vocabulary
        dict(name="adjust_tiny_f32", op="adjust", dtype="f32", requests=4, rows_lo=5, rows_hi=5, vocab=1024, pad=0,
             history=64, tree="chain", mask="some", bias=4),
        # the verify rows of a serving batch, half of them under a grammar
        dict(name="adjust_verify_bf16", op="adjust", dtype="bf16", requests=128, rows_lo=5, rows_hi=5, vocab=VOCAB, pad=0,
             history=1024, tree="chain", mask="some", bias=16),
        # long histories, trees, an odd vocabulary and stride
        dict(name="adjust_tree_f32", op="adjust", dtype="f32", requests=24, rows_lo=3, rows_hi=31, vocab=50021, pad=3,
             history=16000, tree="wide", mask="none", bias=300),
        # one request's tree
        dict(name="verify_tree_f32", op="verify", dtype="f32", requests=1, rows_lo=20, rows_hi=20, vocab=32768, pad=0,
             tree="wide"),
        # a batch of trees of up to 50 nodes
        dict(name="verify_tree_bf16", op="verify", dtype="bf16", requests=24, rows_lo=10, rows_hi=50, vocab=VOCAB, pad=0,
             tree="wide"),
        # committed rows of a serving batch: a few tokens each, some requests ending
        dict(name="pages_commit", op="pages", requests=128, rows_lo=1, rows_hi=5, page=16, len_hi=1024),
        # many requests with prompts to store among them
        dict(name="pages_prompts", op="pages", requests=512, rows_lo=0, rows_hi=400, page=64, len_hi=32768),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("attn", "attn", "adjust", "verify", "pages"))
    dtype = rng.choice(("bf16", "f32"))
    tree = rng.choice(("chain", "wide"))
    if op == "attn":
        n = _log_int(rng, 1, 128)
        hi = _log_int(rng, 1, max(2, 60000 // n))
        kv = rng.choice((1, 2, 4, 8))
        group = rng.choice((1, 2, 4, 5, 7, 8))
        rows = _log_int(rng, 1, min(64, max(2, 800 // n)))
        return dict(op=op, dtype=dtype, requests=n, rows_lo=rng.randint(1, rows), rows_hi=rows,
                    len_lo=rng.choice((0, hi // 2, hi)), len_hi=hi, heads=kv * group, kv_heads=kv,
                    dim=rng.choice((64, 128)), page=rng.choice((8, 16, 32, 64, 128)), tree=tree)
    if op == "pages":
        hi = rng.choice((1, 5, 64, 400))
        return dict(op=op, requests=_log_int(rng, 1, 500), rows_lo=rng.randint(0, min(hi, 5)), rows_hi=hi,
                    page=rng.choice((1, 8, 16, 32, 64, 128)), len_hi=_log_int(rng, 16, 8000))
    n = _log_int(rng, 1, 128)
    rows = _log_int(rng, 1, min(50, max(2, 640 // n)))
    c = dict(op=op, dtype=dtype, requests=n, rows_lo=rng.randint(1, rows), rows_hi=rows,
             vocab=min(VOCAB, _log_int(rng, 1000, 200000)), pad=rng.choice((0, 0, 1, 2, 8, 37)), tree=tree)
    if dtype == "f32" and n * rows > 320:
        c["vocab"] = min(c["vocab"], VOCAB // 2)
    if op == "adjust":
        c.update(history=_log_int(rng, 1, 8000), mask=rng.choice(("none", "some", "all")), bias=rng.choice((0, 1, 20, 300)))
    return c


def _spread(lo, hi, n):
    """n whole numbers evenly between lo and hi, both ends among them."""
    return [hi if n == 1 else lo + (hi - lo) * i // (n - 1) for i in range(n)]


def _shuffled(values, g):
    order = torch.randperm(len(values), generator=g).tolist()
    return [values[i] for i in order]


def _int(values, dtype=torch.int32):
    return torch.tensor(values, dtype=dtype, device="cuda")


def _type(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _layout(case, g):
    """Row counts of the requests, and the rows' offsets, owners and parents
    (a parent is a row of the same request, counted from its first; -1 at the
    root)."""
    counts = _shuffled(_spread(case["rows_lo"], case["rows_hi"], case["requests"]), g)
    offsets, owner, parents = [0], [], []
    for i, n in enumerate(counts):
        offsets.append(offsets[-1] + n)
        owner += [i] * n
        for j in range(n):
            back = 1
            if case["tree"] == "wide" and j > 1:
                # drafts in the order of their depth: parents move on slowly
                back = int(torch.randint(1, j // 2 + 2, (1,), generator=g))
            parents.append(j - back if j else -1)
    return dict(counts=counts, offsets=_int(offsets), owner=_int(owner), parents=_int(parents),
                chain=case["tree"] == "chain", rows=offsets[-1], most=max(counts))


def _logits(case, rows, gg):
    x = torch.randn(rows, case["vocab"], device="cuda", generator=gg)
    x *= torch.rand(rows, 1, device="cuda", generator=gg) * 2 + 1
    wide = torch.full((rows, case["vocab"] + case["pad"]), math.nan, dtype=_type(case), device="cuda")
    wide[:, :case["vocab"]] = x
    return wide


def prepare(case, seed):
    g = torch.Generator().manual_seed(seed)
    gg = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(op=case["op"])
    if case["op"] == "pages":
        return _prepare_pages(case, g, s)
    s.update(_layout(case, g))
    if case["op"] == "attn":
        return _prepare_attn(case, g, gg, s)
    b, r, v = case["requests"], s["rows"], case["vocab"]
    s["vocab"] = v
    s["logits"] = x = _logits(case, r, gg)
    first = set(s["offsets"].tolist())
    drafts = torch.randint(0, v, (r,), generator=g)
    if case["op"] == "verify":
        # most rows' arg-max is the draft of one of their children
        par, at, children = s["parents"].tolist(), 0, {}
        for row in range(r):
            at = row if row in first else at
            if row != at:
                children.setdefault(at + par[row], []).append(row)
        top = torch.randint(0, v, (r,), generator=g)
        pick = torch.rand(r, 2, generator=g).tolist()
        for row, below in children.items():
            if pick[row][0] < 0.8:
                top[row] = drafts[below[int(pick[row][1] * len(below))]]
        x.scatter_(1, top.cuda()[:, None], 40.0)
    else:
        _prepare_adjust(case, g, gg, s)
    s["drafts"] = drafts[[row for row in range(r) if row not in first]].to(torch.int32).cuda()
    assert s["drafts"].numel() == r - b
    return s


def _prepare_attn(case, g, gg, s):
    dt, page, dim, kv, b, r = _type(case), case["page"], case["dim"], case["kv_heads"], case["requests"], s["rows"]
    lens = _shuffled(_spread(case["len_lo"], case["len_hi"], b), g)
    used = [-(-n // page) for n in lens]
    pages = sum(used) + 3
    ids = torch.randperm(pages, generator=g).to(torch.int32)
    table = torch.full((b, max(used) + 1), -1, dtype=torch.int32)
    at = 0
    for i, n in enumerate(used):
        table[i, :n] = ids[at:at + n]
        at += n
    s.update(lens=lens, length=_int(lens), table=table.cuda(), scale=dim ** -0.5)
    s["k_cache"] = torch.randn(pages, page, kv, dim, device="cuda", dtype=dt, generator=gg)
    s["v_cache"] = torch.randn(pages, page, kv, dim, device="cuda", dtype=dt, generator=gg)
    # q, k and v as one projection leaves them: slices of the same rows
    qkv = torch.randn(r, case["heads"] + 2 * kv, dim, device="cuda", dtype=dt, generator=gg)
    s["q"], s["k"], s["v"] = qkv.split((case["heads"], kv, kv), 1)
    s["q"] *= 1.5
    return s


def _prepare_adjust(case, g, gg, s):
    b, v, h = case["requests"], case["vocab"], case["history"]
    # few tokens make up most of a text
    s["history"] = (torch.rand(b, h, device="cuda", generator=gg) ** 4 * v).to(torch.int32).clamp(max=v - 1)
    total = _shuffled(_spread(0 if b > 2 else h, h, b), g)
    s["history_len"] = _int(total)
    s["prompt_len"] = _int([n * (i % 4) // 4 for i, n in enumerate(total)])
    pick = torch.arange(b, device="cuda")
    s["repetition"] = torch.tensor((1.0, 1.1, 1.3, 0.9), device="cuda")[pick % 4]
    s["frequency"] = torch.tensor((0.0, 0.5, -0.2), device="cuda")[pick % 3]
    s["presence"] = torch.tensor((0.6, 0.0, 0.0, 0.3, 0.0), device="cuda")[pick % 5]
    s["bias_offsets"] = s["bias_tokens"] = s["bias_values"] = s["mask"] = s["mask_index"] = None
    if case["bias"]:
        n = _shuffled(_spread(0 if b > 1 else case["bias"], case["bias"], b), g)
        s["bias_offsets"] = _int([sum(n[:i]) for i in range(b + 1)])
        s["bias_tokens"] = torch.randint(0, v, (sum(n),), device="cuda", dtype=torch.int32, generator=gg)
        value = torch.rand(sum(n), device="cuda", generator=gg) * 8 - 4
        value[::7] = -math.inf
        s["bias_values"] = value
    if case["mask"] != "none":
        r = s["rows"]
        rows = list(range(r)) if case["mask"] == "all" else list(range(0, r, 2))
        words = torch.randint(-2 ** 31, 2 ** 31, (len(rows), (v + 31) // 32), device="cuda", dtype=torch.int64, generator=gg)
        # every second state of the grammar allows few tokens
        few = torch.randint(-2 ** 31, 2 ** 31, words.shape, device="cuda", dtype=torch.int64, generator=gg)
        words[::2] &= few[::2] & (few[::2] >> 7) & (few[::2] << 5)
        s["mask"] = words.to(torch.int32)
        index = torch.full((r,), -1, dtype=torch.int32)
        index[rows] = torch.arange(len(rows), dtype=torch.int32)
        s["mask_index"] = index.cuda()


def _prepare_pages(case, g, s):
    b, page = case["requests"], case["page"]
    # a request in sixteen has ended and gives its pages back, and one holds
    # more than it needs
    ended = b // 16
    rows = _shuffled(_spread(case["rows_lo"], case["rows_hi"], b - ended) + [0] * ended, g)
    used = _shuffled(_spread(0, case["len_hi"], b), g)
    more = b // 16
    lens, held = [], []
    for i in range(b):
        gone = rows[i] == 0 and ended > 0
        ended -= gone
        lens.append(0 if gone else used[i])
        held.append(-(-used[i] // page) + (2 if more > 0 and not gone else 0))
        more -= more > 0 and not gone
    width = -(-case["len_hi"] // page) + -(-case["rows_hi"] // page) + 4
    grown = sum(-(-n // page) for n in rows) + b
    pool = sum(held) + grown
    ids = torch.randperm(pool, generator=g).to(torch.int32)
    table = torch.full((b, width), -1, dtype=torch.int32)
    at = 0
    for i, n in enumerate(held):
        table[i, :n] = ids[at:at + n]
        at += n
    free = torch.full((pool,), -1, dtype=torch.int32)
    free[:pool - at] = ids[at:]
    offsets = [0]
    for n in rows:
        offsets.append(offsets[-1] + n)
    s.update(page=page, rows=offsets[-1] + 7, table=table.cuda(), held=_int(held), length=_int(lens),
             offsets=_int(offsets), free=free.cuda(), free_count=_int([pool - at]))
    return s


def _plain_attn(s):
    q, k, v, par = s["q"], s["k"], s["v"], s["parents"]
    heads, dim = q.shape[1:]
    kv = k.shape[1]
    out, lse, at = [], [], 0
    for i, (n, length) in enumerate(zip(s["counts"], s["lens"])):
        rows = slice(at, at + n)
        ids = s["table"][i, :-(-length // s["k_cache"].shape[1])].long()
        keys = torch.cat((s["k_cache"][ids].reshape(-1, kv, dim)[:length], k[rows])).float()
        values = torch.cat((s["v_cache"][ids].reshape(-1, kv, dim)[:length], v[rows])).float()
        # a row sees the context, itself and the rows above it
        own_row = torch.arange(n, device=q.device)
        sees = own_row[:, None] == own_row
        up = own_row
        for _ in range(n - 1):
            up = torch.where(up > 0, par[rows].long()[up], up)
            sees = sees | (up[:, None] == own_row)
        sees = torch.cat((torch.ones(n, length, dtype=torch.bool, device=q.device), sees), 1)
        x = q[rows].float().reshape(n, kv, heads // kv, dim).permute(1, 0, 2, 3).reshape(kv, -1, dim)
        score = x @ keys.permute(1, 2, 0).contiguous() * s["scale"]
        score = score.reshape(kv, n, heads // kv, -1).masked_fill(~sees[None, :, None], -math.inf)
        m = score.max(-1, keepdim=True).values
        w = torch.exp(score - m)
        total = w.sum(-1, keepdim=True)
        y = (w / total).reshape(kv, n * (heads // kv), -1) @ values.permute(1, 0, 2).contiguous()
        out.append(y.reshape(kv, n, heads // kv, dim).permute(1, 0, 2, 3).reshape(n, heads, dim))
        lse.append((m + torch.log(total))[..., 0].permute(1, 0, 2).reshape(n, heads))
        at += n
    return {"out": torch.cat(out).to(q.dtype), "lse": torch.cat(lse)}


def _plain_row_tokens(s):
    """Draft of every row (-1 at a root), and every row's parent as a row of
    the batch."""
    r = s["rows"]
    start = s["offsets"].long()[s["owner"].long()]
    row = torch.arange(r, device=start.device)
    root = row == start
    token = torch.full((r,), -1, dtype=torch.int64, device=start.device)
    token = torch.where(root, token, s["drafts"].long()[(row - s["owner"].long() - 1).clamp(0, max(s["drafts"].numel() - 1, 0))]
                        if s["drafts"].numel() else token)
    return token, torch.where(root, row, start + s["parents"].long())


def _plain_adjust(s):
    x = s["logits"][:, :s["vocab"]].float()
    r, v = x.shape
    owner = s["owner"].long()
    at = torch.arange(s["history"].shape[1], device=x.device)
    used = at < s["history_len"].long()[:, None]
    put = used & (at >= s["prompt_len"].long()[:, None])
    tokens = s["history"].long()[owner]
    seen = torch.zeros_like(x).scatter_add_(1, tokens, used[owner].float())
    count = torch.zeros_like(x).scatter_add_(1, tokens, put[owner].float())
    token, up = _plain_row_tokens(s)
    at = torch.arange(r, device=x.device)
    for _ in range(s["most"] - 1):
        one = (token[at] >= 0).float()[:, None]
        count.scatter_add_(1, token[at].clamp(min=0)[:, None], one)
        at = up[at]
    seen = (seen + count) > 0
    per = {k: s[k][owner][:, None] for k in ("repetition", "frequency", "presence")}
    y = torch.where(seen, torch.where(x > 0, x / per["repetition"], x * per["repetition"]), x)
    y = y - per["frequency"] * count
    y = torch.where(count > 0, y - per["presence"], y)
    if s["bias_offsets"] is not None:
        # a token named twice has the value of its last entry
        n = s["bias_tokens"].numel()
        entry = torch.arange(n, device=x.device)
        of = torch.searchsorted(s["bias_offsets"].long(), entry, right=True) - 1
        b = s["bias_offsets"].numel() - 1
        last = torch.full((b * v,), -1, device=x.device).scatter_reduce(0, of * v + s["bias_tokens"].long(), entry, "amax")
        add = torch.where(last >= 0, s["bias_values"][last.clamp(min=0)], 0.0).reshape(b, v)
        y = y + add[owner]
    if s["mask"] is not None:
        ids = torch.arange(v, device=x.device)
        index = s["mask_index"].long()
        bit = (s["mask"][index.clamp(min=0)][:, ids // 32] >> (ids % 32).int()) & 1
        y = torch.where((bit == 0) & (index >= 0)[:, None], -math.inf, y)
    return {"logits": y.to(s["logits"].dtype)}


def _plain_verify(s):
    x = s["logits"][:, :s["vocab"]].float()
    r, v = x.shape
    m = x.max(1, keepdim=True).values
    best = torch.where(x == m, torch.arange(v, device=x.device), v).min(1).values
    lse = m[:, 0] + torch.log(torch.exp(x - m).sum(1))
    token, up = _plain_row_tokens(s)
    owner, b = s["owner"].long(), s["offsets"].numel() - 1
    row = torch.arange(r, device=x.device)
    at = s["offsets"].long()[:-1]
    accepted = torch.zeros_like(at)
    path, steps = [at], [at >= 0]
    for _ in range(s["most"] - 1):
        fits = (token == best[at][owner]) & (up == at[owner]) & (token >= 0)
        child = torch.full_like(at, r).scatter_reduce(0, owner, torch.where(fits, row, r), "amin")
        go = child < r
        at = torch.where(go, child, at)
        accepted = accepted + go
        path.append(at)
        steps.append(go)
    nxt = best[at]
    offsets = torch.cat((accepted.new_zeros(1), torch.cumsum(accepted + 1, 0)))
    rows = torch.full((r + 1,), -1, dtype=torch.int64, device=x.device)
    tokens = rows.clone()
    for j, (where, there) in enumerate(zip(path, steps)):
        rows[torch.where(there, offsets[:-1] + j, r)] = where
        if j:
            tokens[torch.where(there, offsets[:-1] + j - 1, r)] = token[where]
    tokens[offsets[:-1] + accepted] = nxt
    out = dict(accepted_len=accepted, next_token=nxt, out_offsets=offsets, out_tokens=tokens[:r], out_rows=rows[:r],
               row_token=best)
    return {**{k: t.to(torch.int32) for k, t in out.items()}, "row_lse": lse}


def _plain_pages(s):
    page, table, free, r = s["page"], s["table"], s["free"].long(), s["rows"]
    dev = table.device
    off, held, length = s["offsets"].long(), s["held"].long(), s["length"].long()
    n = off[1:] - off[:-1]
    need = (length + n + page - 1) // page
    back, take = (held - need).clamp(min=0), (need - held).clamp(min=0)
    at = torch.arange(table.shape[1], device=dev)
    gives = (at >= need[:, None]) & (at < held[:, None])
    place = s["free_count"].long() + (torch.cumsum(back, 0) - back)[:, None] + at - need[:, None]
    size = free.numel()
    free = torch.cat((free, free[:1])).scatter(0, torch.where(gives, place, size).reshape(-1), table.long().reshape(-1))[:size]
    top = s["free_count"].long() + back.sum()
    takes = (at >= held[:, None]) & (at < need[:, None])
    place = top - 1 - ((torch.cumsum(take, 0) - take)[:, None] + at - held[:, None])
    table = torch.where(takes, free[place.clamp(0, size - 1)], table.long())
    row = torch.arange(r, device=dev)
    of = (torch.searchsorted(off, row, right=True) - 1).clamp(max=n.numel() - 1)
    inside = row < off[-1]
    pos = torch.where(inside, length[of] + row - off[of], -1)
    slot = table[of, (pos // page).clamp(0, table.shape[1] - 1)] * page + pos % page
    return {"slot": torch.where(inside, slot, -1), "position": pos.to(torch.int32), "length": (length + n).to(torch.int32),
            "held": need.to(torch.int32), "free_count": (top - take.sum()).to(torch.int32),
            "block_table": table.to(torch.int32), "free_pages": free.to(torch.int32)}


def _own(s):
    import draft_token_verification_packed_amd as vsv
    if s["op"] == "pages":
        out = vsv.plan_pages(s["table"], s["held"], s["length"], s["offsets"], s["free"], s["free_count"], s["page"],
                             num_rows=s["rows"])
        return {**{k: out[k] for k in ("slot", "position", "length", "held", "free_count")}, "block_table": s["table"],
                "free_pages": s["free"]}
    parents = None if s["chain"] else s["parents"]
    if s["op"] == "attn":
        out, lse = vsv.tree_attention(s["q"], s["k"], s["v"], s["offsets"], s["k_cache"], s["v_cache"], s["table"],
                                      s["length"], parents=parents, scale=s["scale"], return_lse=True)
        return {"out": out, "lse": lse}
    if s["op"] == "adjust":
        return {"logits": vsv.adjust_logits(
            s["logits"], s["offsets"], s["drafts"], parents=parents, history=s["history"], history_len=s["history_len"],
            prompt_len=s["prompt_len"], repetition=s["repetition"], frequency=s["frequency"], presence=s["presence"],
            bias_offsets=s["bias_offsets"], bias_tokens=s["bias_tokens"], bias_values=s["bias_values"], mask=s["mask"],
            mask_index=s["mask_index"], vocab=s["vocab"])}
    out = vsv.verify_greedy_tree(s["logits"], s["offsets"], s["owner"], s["drafts"], s["parents"], vocab=s["vocab"])
    return {k: out[k] for k in ("accepted_len", "next_token", "out_offsets", "out_tokens", "out_rows", "row_token",
                                "row_lse")}


def run(state):
    if own:
        return _own(state)
    return {"attn": _plain_attn, "adjust": _plain_adjust, "verify": _plain_verify, "pages": _plain_pages}[state["op"]](state)


def work(case):
    b = case["requests"]
    counts = _spread(case["rows_lo"], case["rows_hi"], b)
    rows = sum(counts)
    if case["op"] == "pages":
        return {"bytes": 16 * b + 4 * b * 2 + 12 * rows + 8 * rows // case["page"], "flops": 4 * rows}
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "attn":
        lens = _spread(case["len_lo"], case["len_hi"], b)
        heads, kv, dim = case["heads"], case["kv_heads"], case["dim"]
        n, most = sum(lens), case["rows_hi"]
        # rows and lengths are paired by chance: the mean of every pairing
        pairs = sum(counts) * n / b + sum(c * (c + 1) / 2 for c in counts)
        return {"bytes": 2 * n * kv * dim * e + rows * (2 * heads + 2 * kv) * dim * e + 4 * rows * heads
                + 4 * (n // case["page"] + 2 * b + min(rows, most * b)), "flops": int(4 * dim * heads * pairs)}
    v = case["vocab"]
    if case["op"] == "verify":
        return {"bytes": rows * v * e + 32 * rows, "flops": 3 * rows * v}
    masked = {"none": 0, "some": (rows + 1) // 2, "all": rows}[case["mask"]]
    small = 4 * sum(_spread(0 if b > 2 else case["history"], case["history"], b)) + 4 * b * case["bias"]
    return {"bytes": 2 * rows * v * e + masked * ((v + 31) // 32) * 4 + small, "flops": 4 * rows * v}


def _paths(s):
    """For every row of the batch, the rows from its root to itself."""
    off, par = s["offsets"].tolist(), s["parents"].tolist()
    paths = []
    for i in range(len(off) - 1):
        for r in range(off[i], off[i + 1]):
            paths.append([r] if r == off[i] else paths[off[i] + par[r]] + [r])
    return paths


def _exact_attn(s):
    q, paths, off = s["q"].double(), _paths(s), s["offsets"].tolist()
    heads, kv = q.shape[1], s["k"].shape[1]
    out, lse = torch.zeros_like(q), torch.zeros(q.shape[:2], dtype=torch.float64, device=q.device)
    page = s["k_cache"].shape[1]
    for i, length in enumerate(s["lens"]):
        first, n = off[i], off[i + 1] - off[i]
        bias = torch.full((n, length + n), -math.inf, dtype=torch.float64)
        bias[:, :length] = 0
        for j in range(n):
            bias[j, [length + r - first for r in paths[first + j]]] = 0
        bias = bias.to(q.device)
        token = torch.arange(length, device=q.device)
        where = (s["table"][i].long()[token // page], token % page)
        for h in range(kv):
            keys = torch.cat((s["k_cache"][where[0], where[1], h], s["k"][first:first + n, h])).double()
            values = torch.cat((s["v_cache"][where[0], where[1], h], s["v"][first:first + n, h])).double()
            for a in range(h * heads // kv, (h + 1) * heads // kv):
                score = torch.mm(q[first:first + n, a], keys.t()) * s["scale"] + bias
                lse[first:first + n, a] = torch.logsumexp(score, 1)
                out[first:first + n, a] = torch.mm(torch.softmax(score, 1), values)
    return {"out": out, "lse": lse}


def _exact_adjust(s):
    v, paths, first, owner = s["vocab"], _paths(s), s["offsets"].tolist(), s["owner"].tolist()
    out = s["logits"][:, :v].double()
    drafts = s["drafts"].tolist()
    host = {k: s[k].double().tolist() for k in ("repetition", "frequency", "presence")}
    for r in range(out.shape[0]):
        i = owner[r]
        x = out[r]
        text = s["history"][i].long()
        end, prompt = int(s["history_len"][i]), int(s["prompt_len"][i])
        ahead = torch.tensor([drafts[p - i - 1] for p in paths[r] if p != first[i]], dtype=torch.int64, device=x.device)
        written = torch.cat((text[prompt:end], ahead))
        count = torch.bincount(written, minlength=v).double()
        seen = (count + torch.bincount(text[:prompt], minlength=v)) > 0
        rho = host["repetition"][i]
        x = torch.where(seen & (x > 0), x / rho, torch.where(seen, x * rho, x))
        x = x - host["frequency"][i] * count - host["presence"][i] * (count > 0)
        if s["bias_offsets"] is not None:
            b0, b1 = s["bias_offsets"][i].item(), s["bias_offsets"][i + 1].item()
            named = dict(zip(s["bias_tokens"][b0:b1].tolist(), s["bias_values"][b0:b1].tolist()))
            ids = torch.tensor(list(named), dtype=torch.int64, device=x.device)
            x[ids] += torch.tensor(list(named.values()), dtype=torch.float64, device=x.device)
        if s["mask"] is not None and s["mask_index"][r] >= 0:
            words = s["mask"][s["mask_index"][r].item()].long() & 0xFFFFFFFF
            bits = (words[:, None] >> torch.arange(32, device=x.device)) & 1
            x[bits.reshape(-1)[:v] == 0] = -math.inf
        out[r] = x
    return {"logits": out}


def _exact_verify(s):
    v, off, par = s["vocab"], s["offsets"].tolist(), s["parents"].tolist()
    x = s["logits"][:, :v].double()
    lse = torch.logsumexp(x, 1)
    best = [int((row == row.max()).nonzero()[0]) for row in x]
    drafts = s["drafts"].tolist()
    o = dict(accepted_len=[], next_token=[], out_offsets=[0], out_tokens=[], out_rows=[], row_token=best)
    for i in range(len(off) - 1):
        at = off[i]
        steps = [at]
        while True:
            below = [r for r in range(at + 1, off[i + 1]) if off[i] + par[r] == at and drafts[r - i - 1] == best[at]]
            if not below:
                break
            at = below[0]
            steps.append(at)
        o["accepted_len"].append(len(steps) - 1)
        o["next_token"].append(best[at])
        o["out_tokens"] += [drafts[r - i - 1] for r in steps[1:]] + [best[at]]
        o["out_rows"] += steps
        o["out_offsets"].append(len(o["out_rows"]))
    for k in ("out_tokens", "out_rows"):
        o[k] += [-1] * (len(best) - len(o[k]))
    return {**{k: torch.tensor(t, dtype=torch.int32) for k, t in o.items()}, "row_lse": lse}


def _exact_pages(s):
    page, off = s["page"], s["offsets"].tolist()
    table, held, length = s["table"].tolist(), s["held"].tolist(), s["length"].tolist()
    stack = s["free"].tolist()
    top = s["free_count"].item()
    need = [-(-(n + off[i + 1] - off[i]) // page) for i, n in enumerate(length)]
    for i in range(len(need)):
        for p in range(need[i], held[i]):
            stack[top] = table[i][p]
            top += 1
    slot, position = [], []
    for i in range(len(need)):
        for p in range(held[i], need[i]):
            top -= 1
            table[i][p] = stack[top]
        for j in range(off[i + 1] - off[i]):
            p = length[i] + j
            position.append(p)
            slot.append(table[i][p // page] * page + p % page)
    more = [-1] * (s["rows"] - off[-1])
    total = [n + off[i + 1] - off[i] for i, n in enumerate(length)]
    t32 = lambda a: torch.tensor(a, dtype=torch.int32)
    return {"slot": torch.tensor(slot + more), "position": t32(position + more), "length": t32(total), "held": t32(need),
            "free_count": t32([top]), "block_table": t32(table), "free_pages": t32(stack)}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("adjust", "verify") and s["rows"] * case["vocab"] > 200_000_000:
        return None  # over a few GB in 64 bits
    if case["op"] == "attn" and s["rows"] * case["heads"] * max(s["lens"]) > 400_000_000:
        return None
    return {"attn": _exact_attn, "adjust": _exact_adjust, "verify": _exact_verify, "pages": _exact_pages}[case["op"]](s)
