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
