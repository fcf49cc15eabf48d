"""AdamW where a factor of its update comes near the end of fp32's bits: decays
far below a weight's last bit."""
import math

import pytest
import torch

import ssim_loss_amd as S
from gpu_util import say
from train_oracle import U, adamw, check

pytestmark = pytest.mark.gpu


# (one launch, and two)
@pytest.mark.parametrize("n", [5000, 50_000])
@pytest.mark.parametrize("lr", [1e-4, 1e-5, 1e-6])
@pytest.mark.parametrize("grads", [True, False])
def test_decay_far_below_a_weights_last_bit(lr, n, grads):
    """lr weight_decay of 1e-6 to 1e-8, beside steps of a like size: the new
    weight is the exact one but for its own rounding (half a step) and the few
    of the change that is taken from it."""
    say("decay", lr, n, grads)
    decay, b1, b2, eps, t = 0.01, 0.9, 0.99, 1.0, 5
    rng = torch.Generator(device="cuda").manual_seed(90)
    w = torch.randn(n, generator=rng, device="cuda") + 3.0
    g = torch.randn(n, generator=rng, device="cuda") * (decay if grads else 0.0)
    m, v = torch.zeros_like(w), torch.zeros_like(w)
    before = [x.cpu() for x in (w, m, v, g)]
    opt = S.AdamW([w], lr=lr, betas=(b1, b2), eps=eps, weight_decay=decay, exp_avgs=[m],
                  exp_avg_sqs=[v], step=t - 1)
    opt.step([g])
    (want, _), _, (m1, _), (v1, _) = adamw(before[0], None, *before[1:], 1.0, lr, b1, b2, eps, decay, t)
    step = lr / (1 - b1 ** t) * m1 / ((v1 / (1 - b2 ** t)).sqrt() + eps)
    # the change: its two terms (the step's: 6 of m, 8 of the root, eps, sum, quotient, size, product) and their sum
    change = 20 * U * (step.abs() + lr * decay * before[0].double().abs())
    check(w, want, want.abs() * U + change, "weights")


def test_decay_of_weights_that_are_not_finite():
    w = torch.tensor([math.inf, -math.inf, math.nan, 1.0] * 3, device="cuda")
    opt = S.AdamW([w], lr=1e-3, weight_decay=0.0)
    for decay in (0.0, 0.1):
        opt.weight_decay = decay
        opt.step([torch.zeros_like(w)])
        assert (w[0::4] == math.inf).all() and (w[1::4] == -math.inf).all() and torch.isnan(w[2::4]).all()
        assert torch.isfinite(w[3::4]).all()
