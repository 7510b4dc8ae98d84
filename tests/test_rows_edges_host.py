"""Refusals of the row operators at the edges of what they accept. Needs no
GPU."""
import pytest
import torch

import draft_token_verification_packed_amd as vsv


def test_forward_mode_is_refused():
    # a dual tensor does not require a gradient, and its tangent would be lost
    import torch.autograd.forward_ad as fw
    x, i, f = torch.zeros(4, 16), torch.zeros(4, 1, dtype=torch.int32), torch.zeros(4, 1)
    with fw.dual_level():
        dual = fw.make_dual(x, torch.ones(4, 16))
        for student in (dual, dual * 2.0):
            with pytest.raises(NotImplementedError):
                vsv.distill_loss(student, i, f)
            with pytest.raises(NotImplementedError):
                vsv.distill_loss(student, i, f, vocab=15)
        with pytest.raises(ValueError):          # a plain host tensor: refused as that
            vsv.distill_loss(x, i, f)


def test_error_words_outlive_inference_mode(monkeypatch):
    # words are cut from a block that many calls share: one made under
    # inference mode would be refused in place by a later caller outside it
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    monkeypatch.setattr(vsv, "_flag_words", {})
    cpu = torch.device("cpu")
    with torch.inference_mode():
        first = vsv._new_flag(cpu, 0)
        first.zero_()
    word = vsv._new_flag(cpu, 0)
    assert word.data_ptr() == first.data_ptr() + 4
    assert not word.is_inference()
    word.fill_(3)
    first.zero_()
    assert int(word) == 3 and int(first) == 0


@pytest.mark.parametrize("T", [1.4e-45, 1e-40, 4.2e-39])
def test_temperatures_without_a_reciprocal_are_refused(T):
    # log2(e) / T is beyond float32 there, and 0 / T would come out as NaN
    import ctypes
    import os
    if not os.path.exists(vsv.LIB_PATH):
        pytest.skip("library not built (run the package build first)")
    L, P = vsv.lib(), ctypes.c_void_p
    assert L.vsv_top_logits(P(0x10000), 1, 1024, 1024, 4, 8, T, P(8), P(8), None, None, None, 0, None) == 1
    d = vsv.Distill(0x10000, 1, 1024, 1024, 4, 8, 8, 8, None, T)
    assert L.vsv_distill_forward(ctypes.byref(d), P(8), None, None, None, 0, None) == 1
    assert L.vsv_distill_backward(ctypes.byref(d), P(8), None, P(0x20000), 1024, None) == 1
    assert L.vsv_distill_grad(ctypes.byref(d), None, P(8), P(0x20000), 1024, None, None, 0, None) == 1
