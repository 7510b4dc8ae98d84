"""The tree operators as a serving loop uses them: attention, logits,
adjustment, verification, page plan and storing the accepted rows, round after
round without a host read-back; on a side stream, in a captured graph, and
two calls at once."""
import numpy as np
import pytest

import oracle
from tests.tree_cases import layout
from tests.workloads import cuda_or_skip, host, to_dev

pytestmark = pytest.mark.gpu

B, H, KV, D, V, PAGE, WIDTH = 5, 4, 2, 64, 211, 8, 12


@pytest.fixture(scope="module")
def vsv():
    cuda_or_skip()
    import draft_token_verification_packed_amd as m
    m.lib()
    return m


def _model(seed):
    import torch
    g = torch.Generator().manual_seed(seed)
    f = lambda *s: torch.randn(*s, generator=g)
    return {k: t.cuda() for k, t in dict(embed=f(V, 96), place=f(WIDTH * PAGE + 64, 96) * 0.3, qkv=f(96, (H + 2 * KV) * D) * 0.1,
                                         head=f(H * D, V) * 0.5).items()}


def _forward(vsv, m, tokens, where, off, kc, vc, table, length, par):
    """Logits and the rows' keys and values of packed rows."""
    x = m["embed"][tokens.long()] + m["place"][where.long()]
    qkv = (x @ m["qkv"]).view(-1, H + 2 * KV, D)
    q, k, v = qkv.split((H, KV, KV), 1)
    return vsv.tree_attention(q, k, v, off, kc, vc, table, length, par).reshape(-1, H * D) @ m["head"], k, v


def test_rounds_of_tree_verification(vsv):
    """Tokens of the loop equal those of greedy decoding one token at a time
    with a plain cache and the oracle's adjustments."""
    import torch
    m, rng = _model(0), np.random.default_rng(1)
    prompts = [rng.integers(0, V, n) for n in (3, 9, 1, 16, 6)]
    kc = torch.full((B * WIDTH + 3, PAGE, KV, D), float("nan"), device="cuda")
    vc = torch.full_like(kc, float("nan"))
    pool = to_dev(rng.permutation(B * WIDTH + 3).astype(np.int32))
    table = torch.full((B, WIDTH), -1, dtype=torch.int32, device="cuda")
    count = to_dev(np.array([B * WIDTH + 3], dtype=np.int32))
    held, length = [torch.zeros(B, dtype=torch.int32, device="cuda") for _ in range(2)]
    history = torch.zeros((B, 200), dtype=torch.int32, device="cuda")
    prompt_len = to_dev(np.array([len(p) for p in prompts], dtype=np.int32))
    rep = to_dev(np.array([1.3, 1.0, 0.8, 1.1, 1.0], dtype=np.float32))
    pres = to_dev(np.array([0.5, 0.0, 0.3, 0.0, 1.0], dtype=np.float32))
    allowed = rng.random((B, V)) < 0.8
    words = np.zeros((B, (V + 31) // 32 * 32), dtype=np.uint8)
    words[:, :V] = allowed
    mask = to_dev(np.packbits(words, axis=1, bitorder="little").view(np.int32))

    def store(k, v, plan, rows, flat):
        # what an engine's own cache write does with the slots
        keep = plan["slot"] >= 0
        kc.view(-1, KV, D)[plan["slot"][keep]] = k[rows.long()[keep]]
        vc.view(-1, KV, D)[plan["slot"][keep]] = v[rows.long()[keep]]

    # the prompts but their last tokens are stored first (no rows attend)
    fill = [len(p) - 1 for p in prompts]
    off = to_dev(np.concatenate(([0], np.cumsum(fill))).astype(np.int32))
    tokens = to_dev(np.concatenate([p[:-1] for p in prompts]).astype(np.int32))
    plan = vsv.plan_pages(table, held, length, off, pool, count, PAGE, int(sum(fill)))
    x = m["embed"][tokens.long()] + m["place"][plan["position"].long()]
    _, k, v = (x @ m["qkv"]).view(-1, H + 2 * KV, D).split((H, KV, KV), 1)
    store(k, v, plan, torch.arange(sum(fill), device="cuda"), None)
    held, length, count = plan["held"], plan["length"], plan["free_count"]
    for i, p in enumerate(prompts):
        history[i, :len(p)] = to_dev(p.astype(np.int32))
    text = prompt_len.clone()
    last = to_dev(np.array([p[-1] for p in prompts], dtype=np.int32))

    # greedy decoding, one token at a time, in float64 on the host
    W = {k: t.double().cpu().numpy() for k, t in m.items()}
    def decode(i, steps):
        seq = [int(t) for t in prompts[i]]
        margin = np.inf
        for _ in range(steps):
            x = W["embed"][seq] + W["place"][np.arange(len(seq))]
            q, k, v = np.split((x @ W["qkv"]).reshape(len(seq), -1, D), (H, H + KV), 1)
            o = []
            for h in range(H):
                s = k[:, h // 2] @ q[-1, h] * D ** -0.5
                w = np.exp(s - s.max())
                o.append(w @ v[:, h // 2] / w.sum())
            z = oracle.adjust_row(np.concatenate(o) @ W["head"], seq[:len(prompts[i])], seq[len(prompts[i]):],
                                  float(host(rep)[i]), 0.0, float(host(pres)[i]), allowed=allowed[i])
            top = np.sort(z)[-2:]
            margin = min(margin, top[1] - top[0])
            seq.append(int(z.argmax()))
        return seq[len(prompts[i]):], margin
    want = [decode(i, 24) for i in range(B)]
    # the inputs are such that float32 cannot turn an arg-max
    assert min(mg for _, mg in want) > 1e-3

    got = [[] for _ in range(B)]
    for step in range(4):
        counts = rng.integers(1, 12, B)
        o, owner, par = layout(rng, counts)
        drafts = np.zeros(int(o[-1]) - B, dtype=np.int32)
        for i in range(B):
            done = len(got[i])
            for j in range(1, counts[i]):
                # mostly the right token for the row's depth, so that paths are accepted
                depth = len(oracle.path_of(par[o[i]:o[i + 1]], j)) - 1
                drafts[o[i] - i + j - 1] = want[i][0][done + depth - 1] if rng.random() < 0.7 else rng.integers(V)
        R = int(o[-1])
        depth = np.concatenate([[len(oracle.path_of(par[o[i]:o[i + 1]], j)) - 1 for j in range(counts[i])] for i in range(B)])
        d_off, d_owner, d_par, d_drafts = to_dev(o), to_dev(owner), to_dev(par), to_dev(drafts)
        is_root = to_dev(np.isin(np.arange(R), o[:-1]))
        tok = torch.empty(R, dtype=torch.int32, device="cuda")
        tok[is_root] = last
        tok[~is_root] = d_drafts
        where = length[d_owner.long()] + to_dev(depth.astype(np.int32))
        z, k, v = _forward(vsv, m, tok, where, d_off, kc, vc, table, length, d_par)
        z = vsv.adjust_logits(z, d_off, d_drafts, parents=d_par, history=history, history_len=text, prompt_len=prompt_len,
                              repetition=rep, presence=pres, mask=mask, mask_index=d_owner, out=z)
        out = vsv.verify_greedy_tree(z, d_off, d_owner, d_drafts, d_par)
        plan = vsv.plan_pages(table, held, length, out["out_offsets"], pool, count, PAGE, R)
        store(k, v, plan, out["out_rows"], None)
        held, length, count, last = plan["held"], plan["length"], plan["free_count"], out["next_token"]
        for f in (out["error_flag"], plan["error_flag"]):
            assert int(host(f)[0]) == 0
        oo, toks = host(out["out_offsets"]), host(out["out_tokens"])
        for i in range(B):
            new = toks[oo[i]:oo[i + 1]].tolist()
            n = int(text[i])
            history[i, n:n + len(new)] = to_dev(np.array(new, dtype=np.int32))
            got[i] += new
        text = text + out["accepted_len"] + 1
        assert np.array_equal(host(length), host(text) - 1)
    for i in range(B):
        n = min(len(got[i]), 24)
        assert got[i][:n] == want[i][0][:n], i
    assert sum(len(g) for g in got) > 4 * B      # drafts were accepted


def _inputs(seed, dtype="f32"):
    import torch
    rng = np.random.default_rng(seed)
    counts = rng.integers(1, 9, 6)
    off, owner, par = layout(rng, counts)
    R = int(off[-1])
    g = torch.Generator(device="cuda").manual_seed(seed)
    f = lambda *s: torch.randn(*s, device="cuda", generator=g)
    pages = 40
    return dict(off=to_dev(off), owner=to_dev(owner), par=to_dev(par), q=f(R, H, D), k=f(R, KV, D), v=f(R, KV, D),
                kc=f(pages, PAGE, KV, D), vc=f(pages, PAGE, KV, D), R=R,
                table=to_dev(rng.permutation(pages)[:36].reshape(6, 6).astype(np.int32)),
                length=to_dev(rng.integers(0, 6 * PAGE + 1, 6).astype(np.int32)), logits=f(R, V),
                drafts=to_dev(rng.integers(0, 5, R - 6).astype(np.int32)),
                history=to_dev(rng.integers(0, V, (6, 30)).astype(np.int32)),
                used=to_dev(rng.integers(0, 31, 6).astype(np.int32)), rep=f(6).abs() + 0.5,
                pool=to_dev(np.arange(100, 180, dtype=np.int32)), count=to_dev(np.array([80], dtype=np.int32)),
                held=to_dev(np.full(6, 2, dtype=np.int32)), plan_table=to_dev(np.arange(120, dtype=np.int32).reshape(6, 20)),
                stored=to_dev(rng.integers(0, 30, 6).astype(np.int32)))


def _all(vsv, s, **kw):
    """Every operator once; their outputs in one flat list."""
    out, lse = vsv.tree_attention(s["q"], s["k"], s["v"], s["off"], s["kc"], s["vc"], s["table"], s["length"], s["par"],
                                  return_lse=True, **kw)
    y = vsv.adjust_logits(s["logits"], s["off"], s["drafts"], parents=s["par"], history=s["history"],
                          history_len=s["used"], repetition=s["rep"], **kw)
    ver = vsv.verify_greedy_tree(y, s["off"], s["owner"], s["drafts"], s["par"], **kw)
    plan = vsv.plan_pages(s["plan_table"], s["held"], s["stored"], ver["out_offsets"], s["pool"], s["count"], PAGE, s["R"], **kw)
    return [out, lse, y] + [ver[k] for k in sorted(ver)] + [plan[k] for k in sorted(plan)]


def _same(a, b):
    return all(np.array_equal(host(x.float()), host(y.float()), equal_nan=True) for x, y in zip(a, b))


def test_side_streams_and_two_calls_at_once(vsv):
    import torch
    ins = [_inputs(3), _inputs(4)]
    want = [_all(vsv, s) for s in ins]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ins]
    print("side streams", flush=True)
    got = []
    for _ in range(3):
        got = [_all(vsv, s, stream=st) for s, st in zip(ins, streams)]
    busy = torch.randn(2048, 2048, device="cuda") @ torch.randn(2048, 2048, device="cuda")
    for st in streams:
        st.synchronize()
    for a, b in zip(got, want):
        assert _same(a, b)
    with torch.cuda.stream(streams[0]):
        again = _all(vsv, ins[1])
    streams[0].synchronize()
    assert _same(again, want[1])
    with pytest.raises(ValueError):
        vsv.adjust_logits(ins[0]["logits"], ins[0]["off"], ins[1]["drafts"][:1], stream=streams[0])
    del busy


def test_replays_of_a_captured_graph(vsv):
    import torch
    s, other = _inputs(5), _inputs(6)
    want = _all(vsv, s)
    side = torch.cuda.Stream()
    _all(vsv, s, stream=side)              # the stream's workspace exists before the capture
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    print("capturing the tree operators", flush=True)
    with torch.cuda.graph(g, stream=side):
        outs = _all(vsv, s)
    for rep in range(4):
        for t in outs:
            t.fill_(-3)
        _all(vsv, other)                   # eager work between the replays
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert _same(outs, want), rep
    # inputs that change under the graph
    s["q"].mul_(0.5)
    s["logits"].neg_()
    g.replay()
    torch.cuda.synchronize()
    assert _same(outs, _all(vsv, s))
    del g


def test_two_graphs_replayed_at_once(vsv):
    import torch
    ins = [_inputs(8), _inputs(9)]
    want = [_all(vsv, s) for s in ins]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graphs, outs = [], []
    for s in ins:                          # captured on one stream
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], stream=side):
            outs.append(_all(vsv, s))
    streams = [torch.cuda.Stream() for _ in ins]
    for rep in range(3):
        for o in outs:
            for t in o:
                t.fill_(-3)
        torch.cuda.synchronize()
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        assert all(_same(o, w) for o, w in zip(outs, want)), rep
    del graphs


def test_repeated_calls_agree_to_the_bit(vsv):
    s = _inputs(7)
    first = _all(vsv, s)
    for _ in range(5):
        assert _same(_all(vsv, s), first)
