"""Cases of the operators around verification: drawing drafts, the teacher's top logits, distillation.

`run` computes each operator in its plain form, or (own = True) through the
framework's entry points:
    sample_rows        one token per row after temperature, top-k, top-p and
                       min-p, from given random numbers
    top_logits         the k first logits of every row, with its log-sum-exp
    distill_loss       loss of a student's rows against a teacher's top
                       logits, and its gradient through autograd
    distill_loss_grad  loss and gradient in one call
"""
import math

import torch

own = False

VOCAB = 152064


def listed():
    return [
        # a draft step of a small batch: the draft law itself, no filters
        dict(name="sample_step_bf16", op="sample", dtype="bf16", rows=16, vocab=VOCAB, pad=0, temps="one", top_k=0,
             top_p=1.0, min_p=0.0),
        # the smallest call: a toy vocabulary
        dict(name="sample_tiny_f32", op="sample", dtype="f32", rows=4, vocab=1024, pad=0, temps="mixed", top_k=20,
             top_p=0.9, min_p=0.0),
        # a serving batch with every filter on, greedy and sampled requests mixed
        dict(name="sample_ragged_f32", op="sample", dtype="f32", rows=128, vocab=VOCAB, pad=0, temps="mixed", top_k=50,
             top_p=0.9, min_p=0.05),
        # a large batch with top-p alone
        dict(name="sample_large_bf16", op="sample", dtype="bf16", rows=512, vocab=VOCAB, pad=0, temps="low", top_k=0,
             top_p=0.95, min_p=0.0),
        # the teacher's side: a toy batch, the verified rows of a serving
        # batch, and rows of an odd width and stride with the most logits
        dict(name="top_tiny_f32", op="top", dtype="f32", rows=20, vocab=1024, pad=0, k=8, temperature=1.0),
        dict(name="top_rows_bf16", op="top", dtype="bf16", rows=640, vocab=VOCAB, pad=0, k=64, temperature=1.0),
        dict(name="top_wide_f32", op="top", dtype="f32", rows=96, vocab=20011, pad=2, k=256, temperature=0.7),
        # validation loss of a draft head, with the teacher's rest as a bucket
        dict(name="distill_eval_bf16", op="loss", dtype="bf16", rows=640, vocab=VOCAB, pad=0, k=64, rest=True,
             temperature=1.0),
        # few tokens, an odd vocabulary, the teacher renormalised over its top
        dict(name="distill_eval_f32", op="loss", dtype="f32", rows=37, vocab=20011, pad=1, k=17, rest=False,
             temperature=2.0),
        # a training batch: loss and gradient of every row in one call
        dict(name="distill_grad_bf16", op="grad", dtype="bf16", rows=2048, vocab=VOCAB, pad=0, k=64, rest=True,
             temperature=1.0),
        # training steps through autograd
        dict(name="distill_step_f32", op="step", dtype="f32", rows=128, vocab=32768, pad=0, k=32, rest=False,
             temperature=1.5),
        dict(name="distill_step_bf16", op="step", dtype="bf16", rows=512, vocab=VOCAB, pad=0, k=128, rest=True,
             temperature=1.0),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("sample", "top", "loss", "grad", "step"))
    vocab = min(VOCAB, _log_int(rng, 1000, 200000))
    rows = _log_int(rng, 1, 640 if op != "sample" else 512)
    c = dict(op=op, dtype=rng.choice(("bf16", "f32")), rows=rows, vocab=vocab, pad=rng.choice((0, 0, 1, 2, 8, 37)))
    if op == "sample":
        c.update(temps=rng.choice(("one", "mixed", "low", "high")), top_k=rng.choice((0, 0, 1, rng.randint(2, 1000))),
                 top_p=rng.choice((1.0, rng.uniform(0.3, 0.99))), min_p=rng.choice((0.0, 0.0, rng.uniform(0.001, 0.2))))
    else:
        c.update(k=_log_int(rng, 1, 256), temperature=rng.choice((1.0, 1.0, rng.uniform(0.5, 3.0))))
        if op != "top":
            c.update(rest=rng.random() < 0.5)
    return c


def _rows(case, g):
    """Rows of logits: a bulk with a spread of its own for every row, a few
    raised tokens, and the end of the vocabulary unused; [rows, vocab] of a
    wider matrix where the case pads its rows."""
    n, v = case["rows"], case["vocab"]
    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    x = torch.randn(n, v, device="cuda", generator=g)
    x *= torch.rand(n, 1, device="cuda", generator=g) * 2 + 1
    ids = torch.randint(0, v, (n, 48), device="cuda", generator=g)
    x.scatter_add_(1, ids, torch.rand(n, 48, device="cuda", generator=g) * 6 + 2)
    x[:, v - v // 500:] = -math.inf
    wide = torch.full((n, v + case["pad"]), math.nan, dtype=dt, device="cuda")
    wide[:, :v] = x
    return wide


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    n, v = case["rows"], case["vocab"]
    s = dict(op=case["op"], vocab=v, logits=_rows(case, g))
    if case["op"] == "sample":
        t = dict(one=(1.0,), mixed=(0.0, 0.5, 1.0), low=(0.0, 0.7), high=(1.3, 2.0))[case["temps"]]
        pick = torch.arange(n, device="cuda") % len(t)
        s["temperature"] = torch.tensor(t, device="cuda")[pick]
        s["top_k"] = torch.full((n,), case["top_k"], dtype=torch.int32, device="cuda")
        s["top_p"] = torch.full((n,), case["top_p"], device="cuda")
        s["min_p"] = torch.full((n,), case["min_p"], device="cuda")
        s["uniforms"] = torch.rand(n, device="cuda", generator=g)
    else:
        s["k"], s["temperature"] = case["k"], case["temperature"]
    if case["op"] in ("loss", "grad", "step"):
        # the teacher agrees with the student in part; batches end in padding
        # rows without teacher entries, and some rows have fewer than k
        teacher = s["logits"][:, :v].float() * 0.7 + torch.randn(n, v, device="cuda", generator=g)
        top, ids = torch.topk(teacher, case["k"], dim=1)
        s["teacher_lse"] = torch.logsumexp(teacher / case["temperature"], dim=1) if case["rest"] else None
        ids = ids.to(torch.int32)
        used = torch.full((n, 1), case["k"], device="cuda")
        used[::5] = (case["k"] + 1) // 2
        if n > 8:
            used[n - n // 16 - 1:] = 0
        s["ids"] = ids.masked_fill(torch.arange(case["k"], device="cuda") >= used, -1)
        s["top"] = top
        s["weight"] = torch.rand(n, device="cuda", generator=g) / n
    return s


def _plain_sample(s):
    x = s["logits"][:, :s["vocab"]].double()
    temp = s["temperature"].double()[:, None]
    greedy = temp == 0
    temp = torch.where(greedy, 1.0, temp)
    v, order = torch.sort(x, dim=1, descending=True, stable=True)
    m = v[:, :1]
    z = (v - m) / temp
    w = torch.exp(z)
    every = w.sum(1, keepdim=True)
    rank = torch.arange(x.shape[1], device=x.device)
    top_k = s["top_k"].long()[:, None]
    keep = (rank < top_k) | (top_k <= 0)
    c = torch.cumsum(w * keep, 1)
    before = torch.cat((torch.zeros_like(m), c[:, :-1]), 1)
    top_p = s["top_p"].double()[:, None]
    keep = keep & ((top_p >= 1) | (before < top_p * c[:, -1:]))
    min_p = s["min_p"].double()[:, None]
    keep = keep & ((min_p <= 0) | (z >= torch.log(min_p)))
    c = torch.cumsum(w * keep, 1)
    total = c[:, -1:]
    at = (c <= s["uniforms"].double()[:, None] * total).sum(1, keepdim=True)
    at = torch.where(greedy, 0, at)
    logprob = torch.where(greedy, 0.0, z.gather(1, at) - torch.log(total))
    return {"token": order.gather(1, at)[:, 0].to(torch.int32), "logprob": logprob[:, 0].float(),
            "lse": (m / temp + torch.log(every))[:, 0].float()}


def _plain_top(s):
    x = s["logits"][:, :s["vocab"]].float()
    v, order = torch.sort(x, dim=1, descending=True, stable=True)
    z = x / s["temperature"]
    m = z.max(1, keepdim=True).values
    lse = m[:, 0] + torch.log(torch.exp(z - m).sum(1))
    return {"values": v[:, :s["k"]], "ids": order[:, :s["k"]].to(torch.int32), "lse": lse}


def _plain_teacher(s):
    """(probabilities of the entries, of the rest; 0 where unused), in 64
    bits: the rest is what the entries leave of one."""
    used = s["ids"] >= 0
    z = (s["top"].double() / s["temperature"]).masked_fill(~used, -math.inf)
    if s["teacher_lse"] is not None:
        t = torch.exp(z - s["teacher_lse"].double()[:, None])
        rest = (1 - t.sum(1, keepdim=True)).clamp(min=0) * used.any(1, keepdim=True)
        return t, rest
    m = z.max(1, keepdim=True).values
    t = torch.exp(z - torch.where(m == -math.inf, 0.0, m))
    total = t.sum(1, keepdim=True)
    return t / torch.where(total == 0, 1.0, total), torch.zeros_like(total)


def _plain_distill(s, grad):
    t, rest = _plain_teacher(s)
    ids = s["ids"].long()
    used = ids >= 0
    at = ids.clamp(min=0)
    y = s["logits"][:, :s["vocab"]].float() / s["temperature"]
    y = y - y.max(1, keepdim=True).values
    w = torch.exp(y)
    total = w.sum(1, keepdim=True)
    log_q = (y.gather(1, at) - torch.log(total)).double()
    loss = torch.where(t > 0, t * (torch.log(t.clamp(min=1e-300)) - log_q), 0.0).sum(1)
    named = torch.zeros_like(w).scatter_add_(1, at, used.float()) > 0
    other = w.masked_fill(named, 0.0).sum(1, keepdim=True)
    log_r = torch.log((other / total).double())
    loss = loss + torch.where(rest > 0, rest * (torch.log(rest.clamp(min=1e-300)) - log_r), 0.0)[:, 0]
    if not grad:
        return {"loss": loss.float()}
    every = t.sum(1, keepdim=True) + rest
    scale = torch.where((rest > 0) & (other > 0), every - rest * (total / other).double(), every).float()
    q = w / total
    d = torch.where(named, q * every.float(), q * scale)
    d = d.scatter_add_(1, at, -t.float()) * (s["weight"][:, None] / s["temperature"])
    return {"loss": loss.float(), "grad": d.to(s["logits"].dtype)}


def _own(s):
    import draft_token_verification_packed_amd as vsv
    x, v = s["logits"], s["vocab"]
    if s["op"] == "sample":
        out = vsv.sample_rows(x, s["temperature"], s["top_k"], s["top_p"], s["min_p"], s["uniforms"], vocab=v)
        return {"token": out["token"], "logprob": out["logprob"], "lse": out["lse"]}
    if s["op"] == "top":
        out = vsv.top_logits(x, s["k"], temperature=s["temperature"], vocab=v)
        return {"values": out["values"], "ids": out["ids"], "lse": out["lse"]}
    x = x[:, :v]
    more = dict(teacher_lse=s["teacher_lse"], temperature=s["temperature"])
    if s["op"] == "loss":
        return {"loss": vsv.distill_loss(x, s["ids"], s["top"], **more)}
    if s["op"] == "grad":
        loss, grad = vsv.distill_loss_grad(x, s["ids"], s["top"], s["weight"], **more)
        return {"loss": loss, "grad": grad}
    leaf = x.detach().requires_grad_()
    loss = vsv.distill_loss(leaf, s["ids"], s["top"], **more)
    grad, = torch.autograd.grad(loss, leaf, s["weight"])
    return {"loss": loss.detach(), "grad": grad}


def run(state):
    if own:
        return _own(state)
    if state["op"] == "sample":
        return _plain_sample(state)
    if state["op"] == "top":
        return _plain_top(state)
    return _plain_distill(state, state["op"] != "loss")


def work(case):
    n, v = case["rows"], case["vocab"]
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "sample":
        return {"bytes": n * v * e + n * 32, "flops": 4 * n * v}
    if case["op"] == "top":
        return {"bytes": n * v * e + n * (8 * case["k"] + 4), "flops": 3 * n * v}
    small = n * (8 * case["k"] + 12)
    if case["op"] == "loss":
        return {"bytes": n * v * e + small, "flops": 3 * n * v}
    return {"bytes": 2 * n * v * e + small, "flops": 6 * n * v}


def _exact_sample_row(x, temp, top_k, top_p, min_p, u):
    lse = torch.logsumexp(x / temp if temp > 0 else x, 0)
    if temp == 0:
        return int(x.argmax()), x.new_zeros(()), lse
    ids = torch.argsort(x, descending=True, stable=True)
    if 0 < top_k < ids.numel():
        ids = ids[:top_k]
    p = torch.softmax(x[ids] / temp, 0)
    if top_p < 1:
        ids = ids[:int((torch.cumsum(p, 0) < top_p).sum()) + 1]
    if min_p > 0:
        ids = ids[(x[ids] - x[ids[0]]) / temp >= math.log(min_p)]
    law = torch.log_softmax(x[ids] / temp, 0)
    n = min(int((torch.cumsum(torch.exp(law), 0) <= u).sum()), ids.numel() - 1)
    return int(ids[n]), law[n], lse


def _exact_distill_row(y, ids, z, lse, temp, weight):
    """Loss of one row, and its gradient by the chain rule over the law's
    cells: one for every named token, one for the rest."""
    used = ids >= 0
    ids, z = ids[used], z[used] / temp
    if ids.numel() == 0:
        return y.new_zeros(()), torch.zeros_like(y)
    log_q = torch.log_softmax(y / temp, 0)
    if lse is None:
        log_t, log_rest = torch.log_softmax(z, 0), None
    else:
        log_t = z - lse
        left = 1 - torch.exp(log_t).sum()
        log_rest = torch.log(left) if left > 0 else None
    t = torch.exp(log_t)
    loss = (t * (log_t - log_q[ids])).sum()
    cell = torch.exp(log_q) * t.sum()
    cell = cell.index_add(0, ids, -t)
    if log_rest is not None:
        outside = log_q.index_fill(0, ids, -math.inf)
        log_r = torch.logsumexp(outside, 0)
        loss = loss + torch.exp(log_rest) * (log_rest - log_r)
        cell = cell + torch.exp(log_rest) * (torch.exp(log_q) - torch.exp(outside - log_r))
    return loss, cell * weight / temp


def exact(case, seed):
    s = prepare(case, seed)
    v, n = s["vocab"], case["rows"]
    if n * v > 200_000_000:
        return None  # over a few GB in 64 bits
    if case["op"] == "sample":
        par = [s[k].double().tolist() for k in ("temperature", "top_k", "top_p", "min_p", "uniforms")]
        rows = [_exact_sample_row(s["logits"][r, :v].double(), *(int(p[r]) if i == 1 else p[r] for i, p in enumerate(par)))
                for r in range(n)]
        return {"token": torch.tensor([r[0] for r in rows], dtype=torch.int32), "logprob": torch.stack([r[1] for r in rows]),
                "lse": torch.stack([r[2] for r in rows])}
    if case["op"] == "top":
        x = s["logits"][:, :v].double()
        ids = torch.argsort(x, dim=1, descending=True, stable=True)[:, :s["k"]]
        return {"values": x.gather(1, ids), "ids": ids.to(torch.int32), "lse": torch.logsumexp(x / s["temperature"], 1)}
    rows = [_exact_distill_row(s["logits"][r, :v].double(), s["ids"][r].long(), s["top"][r].double(),
                               None if s["teacher_lse"] is None else s["teacher_lse"][r].double(), s["temperature"],
                               s["weight"][r].double()) for r in range(n)]
    loss = torch.stack([r[0] for r in rows])
    if case["op"] == "loss":
        return {"loss": loss}
    return {"loss": loss, "grad": torch.stack([r[1] for r in rows])}
