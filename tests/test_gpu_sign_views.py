"""Views whose memory holds the values with the other sign, as the imaginary part of
a complex number's conjugate: what a norm or a scaling of them may take, and what
has to turn them first."""
import pytest
import torch

import ssim_loss_amd as S

pytestmark = pytest.mark.gpu


def numbers(*shape, seed=0, dtype=torch.float32):
    return torch.randn(shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").to(dtype)


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
def test_norms_and_clipping_take_them(dtype):
    plain, turned = numbers(300, seed=1, dtype=dtype), numbers(77, seed=2, dtype=dtype)
    want_norm = S.grad_norm([plain, -turned])
    want = [plain.clone(), -turned]
    S.clip_grads_(want, 1.0)
    view = torch._neg_view(turned.clone())
    assert torch.equal(S.grad_norm([plain, view]), want_norm)
    held = [plain.clone(), view]
    assert torch.equal(S.clip_grads_(held, 1.0), want_norm)
    assert torch.equal(held[0], want[0]) and view.is_neg() and torch.equal(view.resolve_neg(), want[1])
    grads = [plain, torch._neg_view(turned)]
    out = [torch.zeros_like(plain), torch._neg_view(torch.zeros_like(turned))]
    S.clip_grads_(grads, 1.0, out=out)
    assert torch.equal(out[1].resolve_neg(), want[1])


def test_clipping_between_signs_is_refused():
    a = numbers(50, seed=3)
    for grad, out in ((torch._neg_view(a), torch.zeros_like(a)), (a, torch._neg_view(torch.zeros_like(a)))):
        with pytest.raises(NotImplementedError, match="sign"):
            S.clip_grads_([grad], 1.0, out=[out])


@pytest.mark.parametrize("which", ["residual", "normed", "both"])
def test_a_gradient_that_arrives_at_the_joint_with_its_sign_turned(which):
    x, branch = numbers(20, 64, seed=4).requires_grad_(True), numbers(20, 64, seed=5).requires_grad_(True)
    post = (1 + 0.1 * numbers(64, seed=6)).requires_grad_(True)
    outs = S.block_norm(x, branch, post_weight=post)
    ups = [numbers(20, 64, seed=7), numbers(20, 64, seed=8)]
    some = {"residual": [0], "normed": [1], "both": [0, 1]}[which]
    leaves = (x, branch, post)
    want = torch.autograd.grad([outs[k] for k in some], leaves, [-ups[k] for k in some], retain_graph=True)
    got = torch.autograd.grad([outs[k] for k in some], leaves, [torch._neg_view(ups[k]) for k in some])
    assert all(torch.equal(a, b) for a, b in zip(got, want))
