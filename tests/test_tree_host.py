"""Refusals of the tree operators: a status, or an exception in the binding,
before anything is enqueued. Needs no GPU."""
import ctypes
import os

import pytest
import torch

import draft_token_verification_packed_amd as vsv
from tests.test_abi_host import _batch, _outs

P = ctypes.c_void_p


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(vsv.LIB_PATH):
        pytest.skip("library not built (run the package build first)")
    return vsv.lib()


@pytest.mark.parametrize("bad,status", [
    (dict(logits=None), 1), (dict(dtype=7), 1), (dict(vocab=0), 1), (dict(ld=1000), 1), (dict(num_rows=3), 1),
    (dict(row_offsets=None), 1), (dict(row_owner=None), 1), (dict(draft_tokens=None), 1), (dict(logits=0x10001), 1),
])
def test_verify_tree_refusals(L, bad, status):
    b, o = _batch(**bad), _outs()
    assert L.vsv_verify_greedy_tree(ctypes.byref(b), P(8), ctypes.byref(o), P(8), P(0x100000), 1 << 20, None) == status


def test_verify_tree_other_refusals(L):
    b = _batch()
    for o in (_outs(accepted_len=None), _outs(out_tokens=None)):
        assert L.vsv_verify_greedy_tree(ctypes.byref(b), P(8), ctypes.byref(o), None, P(0x100000), 1 << 20, None) == 1
    o = _outs()
    assert L.vsv_verify_greedy_tree(None, P(8), ctypes.byref(o), None, P(0x100000), 1 << 20, None) == 1
    assert L.vsv_verify_greedy_tree(ctypes.byref(b), P(8), ctypes.byref(o), None, None, 1 << 20, None) == 3
    assert L.vsv_verify_greedy_tree(ctypes.byref(b), P(8), ctypes.byref(o), None, P(0x100000), 64, None) == 3
    e = _batch(num_requests=0, num_rows=0)
    assert L.vsv_verify_greedy_tree(ctypes.byref(e), None, ctypes.byref(o), None, None, 0, None) == 0


def _adjust(L, **kw):
    a = dict(logits=0x100000, out=0x200000, dtype=1, vocab=1000, ld=1000, out_ld=1000, num_requests=4, num_rows=20,
             row_offsets=8, draft_tokens=8, history=8, history_ld=16, history_width=16, history_len=8, bias_offsets=8,
             bias_tokens=8, bias_values=8, num_bias=3, mask=8, mask_ld=32, num_masks=20)
    a.update(kw)
    return L.vsv_adjust_logits(ctypes.byref(vsv.Adjust(**a)), None, None)


@pytest.mark.parametrize("bad", [
    dict(logits=None), dict(out=None), dict(logits=0x100001), dict(out=0x200001), dict(dtype=0, out=0x200002),
    dict(dtype=3), dict(vocab=0), dict(ld=999), dict(out_ld=999), dict(ld=1 << 62), dict(out_ld=1 << 62),
    dict(vocab=1 << 30, ld=1 << 30, out_ld=1 << 30), dict(num_requests=-1), dict(num_rows=-1), dict(row_offsets=None),
    dict(draft_tokens=None), dict(history_len=None), dict(history_width=-1), dict(history_ld=15),
    dict(history_ld=1 << 62), dict(num_bias=-1), dict(bias_tokens=None), dict(bias_values=None), dict(mask_ld=31),
    dict(num_masks=-1), dict(num_masks=19), dict(mask_ld=1 << 62),
    # outputs that overlap the logits without being them
    dict(out=0x100002), dict(out=0x100000 + 39998), dict(out=0x100000 - 39998), dict(out=0x100000, out_ld=1001),
])
def test_adjust_refusals(L, bad):
    assert _adjust(L, **bad) == 1


def test_adjust_noops_and_null(L):
    assert _adjust(L, num_requests=0, logits=None) == 0
    assert _adjust(L, num_rows=0, logits=None) == 0
    assert L.vsv_adjust_logits(None, None, None) == 1


def _pages(L, **kw):
    a = dict(table=0x1000, ld=8, width=8, held=0x2000, length=0x3000, offsets=0x4000, B=4, R=10, free=0x5000, pool=50,
             count=0x6000, page=16, slot=0x7000, position=0x8000, new_held=0x9000, new_length=0xa000, new_count=0xb000)
    a.update(kw)
    p = lambda k: P(a[k]) if a[k] else None
    return L.vsv_plan_pages(p("table"), a["ld"], a["width"], p("held"), p("length"), p("offsets"), a["B"], a["R"],
                            p("free"), a["pool"], p("count"), a["page"], p("slot"), p("position"), p("new_held"),
                            p("new_length"), p("new_count"), None, None)


@pytest.mark.parametrize("bad", [dict([(k, None)]) for k in ("table", "held", "length", "offsets", "free", "count", "slot",
                                                            "new_held", "new_length", "new_count")] + [
    dict(B=-1), dict(B=8193), dict(R=-1), dict(page=0), dict(pool=0), dict(width=0), dict(ld=7), dict(ld=1 << 62),
    dict(B=8000, width=300000, ld=300000), dict(B=8000, width=250000, ld=250000, pool=1 << 30), dict(new_held=0x2000), dict(new_length=0x3000), dict(new_count=0x6000),
    dict(slot=0x7004)])
def test_pages_refusals(L, bad):
    assert _pages(L, **bad) == 1


def test_binding_refusals():
    cpu = torch.zeros(4, 16)
    i = lambda n: torch.zeros(n, dtype=torch.int32)
    with pytest.raises(ValueError):
        vsv.verify_greedy_tree(cpu, i(2), i(4), i(3), i(4))
    with pytest.raises(ValueError):
        vsv.adjust_logits(cpu, i(2), i(3))
    with pytest.raises(NotImplementedError):
        vsv.adjust_logits(cpu.requires_grad_(), i(2), i(3))
    with pytest.raises(ValueError):
        vsv.plan_pages(i(4).view(1, 4), i(1), i(1), i(2), i(9), i(1), 16, 4)


def _attention(L, ws=0x100000, wsn=1 << 30, **kw):
    a = dict(q=0x1000, k=0x2000, v=0x3000, k_cache=0x4000, v_cache=0x5000, out=0x6000, q_row=1024, q_head=128, k_row=256,
             k_head=128, v_row=256, v_head=128, out_row=1024, out_head=128, cache_page=4096, cache_token=256,
             cache_head=128, dtype=1, head_dim=128, num_heads=8, num_kv_heads=2, num_requests=4, num_rows=20,
             row_offsets=8, length=8, block_table=8, table_ld=16, table_width=16, num_pages=64, page_size=16, scale=0.1)
    a.update(kw)
    return L.vsv_tree_attention(ctypes.byref(vsv.Attention(**a)), None, P(ws) if ws else None, wsn, None)


@pytest.mark.parametrize("bad", [dict([(k, None)]) for k in ("q", "k", "v", "k_cache", "v_cache", "out", "row_offsets",
                                                            "length", "block_table")] +
                         [dict([(k, 0x1008)]) for k in ("q", "k", "v", "k_cache", "v_cache", "out")] +
                         [dict([(k, 4)]) for k in ("q_row", "q_head", "k_row", "k_head", "v_row", "v_head", "out_row",
                                                   "out_head", "cache_page", "cache_token", "cache_head")] +
                         [dict([(k, -8)]) for k in ("q_row", "cache_page")] + [dict([(k, 1 << 62)]) for k in ("k_row", "cache_page")] + [
    dict(dtype=2), dict(head_dim=96), dict(dtype=0, head_dim=256), dict(num_heads=9), dict(num_kv_heads=0),
    dict(num_heads=0), dict(num_heads=131072), dict(num_rows=1 << 28, num_requests=65536), dict(num_requests=-1), dict(num_requests=65537), dict(num_rows=-1), dict(table_ld=15),
    dict(table_ld=1 << 62), dict(table_width=0), dict(num_pages=0), dict(page_size=0), dict(page_size=24),
    dict(table_width=1 << 28, table_ld=1 << 28), dict(table_width=1 << 26, table_ld=1 << 26, num_heads=8192,
                                                       num_kv_heads=8192), dict(scale=0.0), dict(scale=-1.0),
    dict(scale=float("nan")), dict(scale=float("inf")), dict(scale=3e38),
    dict(out_head=64), dict(out_row=64), dict(out_row=0), dict(out_row=512), dict(out_row=128, out_head=2048)])
def test_attention_refusals(L, bad):
    assert _attention(L, **bad) == 1


def test_attention_heads_may_come_first(L):
    # (refused for its scratch alone)
    assert _attention(L, ws=0, out_row=128, out_head=20 * 128) == 3
    assert _attention(L, ws=0, num_heads=1, num_kv_heads=1, out_row=128, out_head=0) == 3


def test_attention_scratch_and_noops(L):
    assert _attention(L, ws=0) == 3
    assert _attention(L, ws=0x100080) == 3
    assert _attention(L, wsn=1000) == 3
    assert _attention(L, num_rows=0, q=None) == 0
    assert _attention(L, num_requests=0, q=None) == 0
    assert L.vsv_tree_attention(None, None, None, 0, None) == 1
    assert L.vsv_tree_attention_workspace_bytes(None) == 0
    assert L.vsv_tree_attention_workspace_bytes(ctypes.byref(vsv.Attention(dtype=5))) == 0
