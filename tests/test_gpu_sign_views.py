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
