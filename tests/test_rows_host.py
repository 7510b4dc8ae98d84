"""The row operators' refusals: a status, or an exception in the binding,
before anything is enqueued. Needs no GPU."""
import ctypes
import os

import pytest
import torch

import draft_token_verification_packed_amd as vsv

P = ctypes.c_void_p


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(vsv.LIB_PATH):
        pytest.skip("library not built (run the package build first)")
    return vsv.lib()


def _sample(L, **kw):
    a = dict(logits=0x10000, dtype=1, vocab=1024, ld=1024, rows=4, temperature=8, top_k=8, top_p=8, min_p=8, uniform=8,
             token=8, ws=0x1000, wsn=1 << 24)
    a.update(kw)
    p = {k: P(a[k]) if a[k] else None for k in ("logits", "temperature", "top_k", "top_p", "min_p", "uniform", "token")}
    return L.vsv_sample_rows(p["logits"], a["dtype"], a["vocab"], a["ld"], a["rows"], p["temperature"], p["top_k"],
                             p["top_p"], p["min_p"], p["uniform"], p["token"], None, None, None, P(a["ws"]) if a["ws"] else None, a["wsn"],
                             None)


BAD_ROWS = [dict(logits=None), dict(logits=0x10001), dict(dtype=0, logits=0x10002), dict(dtype=2), dict(vocab=0),
            dict(ld=1023), dict(vocab=1 << 30, ld=1 << 30), dict(dtype=0, vocab=1 << 29, ld=1 << 29),
            dict(ld=1 << 62), dict(rows=-1)]


@pytest.mark.parametrize("bad", BAD_ROWS + [dict([(k, None)]) for k in
                                            ("temperature", "top_k", "top_p", "min_p", "uniform", "token")])
def test_sample_rows_refusals(L, bad):
    assert _sample(L, **bad) == 1


def test_sample_scratch(L):
    size = L.vsv_sample_workspace_bytes
    assert size(0, 1024, 1) == 0 and size(4, 0, 1) == 0 and size(4, 152064, 9) == 0 and size(4, 1024, 0) == 0
    for dtype in (0, 1):
        need = size(4, 152064, dtype)
        big = dict(dtype=dtype, vocab=152064, ld=152064)
        assert 0 < need < 1 << 24
        assert _sample(L, ws=0, **big) == 3
        assert _sample(L, wsn=need - 1, **big) == 3
        assert _sample(L, ws=0x1008, **big) == 3


def test_top_scratch(L):
    size = L.vsv_top_workspace_bytes
    assert size(0, 152064, 1, 8) == 0 and size(4, 0, 1, 8) == 0 and size(4, 152064, 9, 8) == 0
    assert size(4, 152064, 1, 0) == 0 and size(4, 152064, 1, 257) == 0 and size(4, 1024, 0, 8) == 0
    need = size(4, 152064, 1, 100)
    big = dict(vocab=152064, ld=152064, k=100)
    assert 0 < need < 1 << 24
    assert _top(L, ws=0, **big) == 3
    assert _top(L, wsn=need - 1, **big) == 3
    assert _top(L, ws=0x1008, **big) == 3


def test_no_rows_is_a_noop(L):
    assert _sample(L, rows=0, logits=None) == 0
    assert _top(L, rows=0, logits=None) == 0
    for call in (_forward, _backward, _grad):
        assert call(L, rows=0, logits=None) == 0


def _top(L, **kw):
    a = dict(logits=0x10000, dtype=1, vocab=1024, ld=1024, rows=4, k=8, T=1.0, values=8, ids=8, ws=0x1000, wsn=1 << 24)
    a.update(kw)
    return L.vsv_top_logits(P(a["logits"]) if a["logits"] else None, a["dtype"], a["vocab"], a["ld"], a["rows"], a["k"],
                            a["T"], P(a["values"]) if a["values"] else None, P(a["ids"]) if a["ids"] else None, None,
                            None, P(a["ws"]) if a["ws"] else None, a["wsn"], None)


@pytest.mark.parametrize("bad", BAD_ROWS + [
    dict(k=0), dict(k=-1), dict(k=257), dict(vocab=7, k=8), dict(T=0.0), dict(T=-1.0), dict(T=float("inf")),
    dict(T=float("nan")), dict(values=None), dict(ids=None)])
def test_top_logits_refusals(L, bad):
    assert _top(L, **bad) == 1


def _distill(**kw):
    a = dict(logits=0x10000, dtype=1, vocab=1024, ld=1024, rows=4, K=8, ids=8, top=8, lse=None, T=1.0)
    a.update(kw)
    return vsv.Distill(a["logits"], a["dtype"], a["vocab"], a["ld"], a["rows"], a["K"], a["ids"], a["top"], a["lse"],
                       a["T"])


def _forward(L, loss=8, ws=0x1000, wsn=1 << 20, **kw):
    d = _distill(**kw)
    return L.vsv_distill_forward(ctypes.byref(d), P(loss) if loss else None, None, None, P(ws) if ws else None, wsn, None)


def _backward(L, state=8, grad=0x20000, gld=1024, **kw):
    d = _distill(**kw)
    return L.vsv_distill_backward(ctypes.byref(d), P(state) if state else None, None, P(grad) if grad else None, gld, None)


def _grad(L, loss=8, grad=0x20000, gld=1024, ws=0x1000, wsn=1 << 20, **kw):
    d = _distill(**kw)
    return L.vsv_distill_grad(ctypes.byref(d), None, P(loss) if loss else None, P(grad) if grad else None, gld, None,
                              P(ws) if ws else None, wsn, None)


@pytest.mark.parametrize("bad", BAD_ROWS + [
    dict(K=0), dict(K=257), dict(ids=None), dict(top=None), dict(T=0.0), dict(T=-2.0), dict(T=float("nan")),
    dict(T=float("inf"))])
def test_distill_refusals(L, bad):
    for call in (_forward, _backward, _grad):
        assert call(L, **bad) == 1, call


def test_distill_output_refusals(L):
    assert _forward(L, loss=None) == 1
    assert _grad(L, loss=None) == 1
    assert _backward(L, state=None) == 1
    assert _backward(L, state=0x1004) == 1
    for call in (_backward, _grad):
        assert call(L, grad=None) == 1
        assert call(L, grad=0x20001) == 1
        assert call(L, gld=1023) == 1
    assert L.vsv_distill_forward(None, P(8), None, None, None, 0, None) == 1
    assert L.vsv_distill_backward(None, P(8), None, P(8), 1024, None) == 1
    assert L.vsv_distill_grad(None, None, P(8), P(8), 1024, None, None, 0, None) == 1


def test_distill_scratch(L):
    size = L.vsv_distill_workspace_bytes
    assert size(0, 1024, 1) == 0 and size(-3, 1024, 1) == 0 and size(4, 0, 1) == 0 and size(4, 1024, 9) == 0
    need = size(4, 152064, 1)
    assert need > 0
    big = dict(vocab=152064, ld=152064)
    for call, more in ((_forward, {}), (_grad, dict(gld=152064))):
        assert call(L, ws=0, **big, **more) == 3
        assert call(L, wsn=need - 1, **big, **more) == 3
        assert call(L, ws=0x1004, **big, **more) == 3


def test_binding_refuses_host_tensors():
    x, f, i = torch.zeros(4, 16), torch.zeros(4), torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):
        vsv.sample_rows(x, f, i, f, f, f)
    with pytest.raises(ValueError):
        vsv.top_logits(x, 4)
    with pytest.raises(ValueError):
        vsv.distill_loss(x, i[:, None], f[:, None])
    with pytest.raises(ValueError):
        vsv.distill_loss(x, i[:, None], f[:, None], vocab=17)
