"""The tree operators have no derivative, and say so before anything else."""
import pytest
import torch
from torch.autograd import forward_ad

import draft_token_verification_packed_amd as vsv

i32 = lambda n: torch.zeros(n, dtype=torch.int32)


def _attention(**kw):
    a = dict(q=torch.zeros(3, 2, 64), k=torch.zeros(3, 1, 64), v=torch.zeros(3, 1, 64), k_cache=torch.zeros(2, 16, 1, 64),
             v_cache=torch.zeros(2, 16, 1, 64), out=None)
    a.update({n: f(a[n] if a[n] is not None else torch.zeros(3, 2, 64)) for n, f in kw.items()})
    out = a.pop("out")
    return vsv.tree_attention(a["q"], a["k"], a["v"], i32(2), a["k_cache"], a["v_cache"], i32(2).view(1, 2), i32(1), out=out)


def _adjust(**kw):
    a = dict(logits=torch.zeros(3, 8), repetition=torch.ones(1), frequency=torch.zeros(1), presence=torch.zeros(1),
             bias_values=torch.zeros(2), out=torch.zeros(3, 8))
    a.update({n: f(a[n]) for n, f in kw.items()})
    return vsv.adjust_logits(a.pop("logits"), i32(2), i32(2), bias_offsets=i32(2), bias_tokens=i32(2), **a)


CALLS = [(_attention, n) for n in ("q", "k", "v", "k_cache", "v_cache", "out")] + [
    (_adjust, n) for n in ("logits", "repetition", "frequency", "presence", "bias_values", "out")]


@pytest.mark.parametrize("call,name", CALLS)
def test_backward_is_refused(call, name):
    ask = {name: lambda t: t.requires_grad_()}
    with pytest.raises(NotImplementedError):
        call(**ask)
    # (without gradients the call gets as far as the check of devices)
    with torch.no_grad(), pytest.raises(ValueError):
        call(**ask)


@pytest.mark.parametrize("call,name", CALLS)
def test_forward_is_refused(call, name):
    with forward_ad.dual_level(), torch.no_grad():
        with pytest.raises(NotImplementedError):
            call(**{name: lambda t: forward_ad.make_dual(t, torch.ones_like(t))})
        with pytest.raises(ValueError):
            call()
