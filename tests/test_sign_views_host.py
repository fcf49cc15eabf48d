"""Views whose memory holds the values with the other sign are taken where the sign
does not matter (no GPU needed: what comes next is the refusal of CPU tensors)."""
import pytest
import torch

import ssim_loss_amd as S


def view():
    return torch._neg_view(torch.ones(8))


def test_norm_and_clipping_take_them():
    for call in (lambda: S.grad_norm([view()]), lambda: S.clip_grads_([view()], 1.0),
                 lambda: S.clip_grads_([view()], 1.0, out=[view()])):
        with pytest.raises(TypeError, match="GPU tensor"):
            call()


def test_the_joint_and_the_optimizer_do_not():
    one = torch.ones(2, 8)
    for call in (lambda: S.block_norm(view()[None], one[:1]), lambda: S.block_norm(one[:1], view()[None]),
                 lambda: S.block_norm(one, one, scale=view())):
        with pytest.raises(NotImplementedError, match="sign"):
            call()
