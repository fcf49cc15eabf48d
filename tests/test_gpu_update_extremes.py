"""AdamW and clipping where a factor of theirs comes near the end of fp32's
bits: decays far below a weight's last bit, clipping factors that are
subnormal numbers."""
import math

import pytest
import torch

import ssim_loss_amd as S
from gpu_util import say
from train_oracle import U, adamw, check, check_norm, clipped, factor, norm_of

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


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


# (in one launch, in two, and past the caches)
@pytest.mark.parametrize("n", [3000, 100_000, 30_000_000])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("max_norm", [1.0, 1e-6])
def test_clip_by_a_factor_that_fp32_holds_as_a_subnormal(max_norm, dtype, n):
    say("clip", max_norm, dtype, n)
    rng = torch.Generator(device="cuda").manual_seed(91)
    g = (torch.randn(n, generator=rng, device="cuda") * 3e37).to(dtype)
    g[:4] = torch.tensor([0.0, 1e-30, 1.0, -1e20], device="cuda").to(dtype)
    before = g.cpu()
    norm = norm_of([before])
    c = factor(norm, max_norm)
    got = S.clip_grads_([g], max_norm)
    check_norm(got, norm) if norm < 3e38 else None
    check(g, *clipped(before, c), "gradients")


def test_adamw_of_gradients_whose_factor_is_subnormal():
    rng = torch.Generator(device="cuda").manual_seed(92)
    for n in (3000, 100_000):
        w = torch.randn(n, generator=rng, device="cuda")
        g = torch.randn(n, generator=rng, device="cuda") * 3e37
        m, v = torch.zeros_like(w), torch.zeros_like(w)
        before = [x.cpu() for x in (w, m, v, g)]
        S.AdamW([w], lr=1e-3, betas=(0.9, 0.97), eps=1e-8, weight_decay=0.02, max_norm=1.0, exp_avgs=[m],
                exp_avg_sqs=[v], step=3).step([g])
        c = factor(norm_of([before[3]]), 1.0)
        p, _, m1, v1 = adamw(before[0], None, *before[1:], c, 1e-3, 0.9, 0.97, 1e-8, 0.02, 4)
        check(w, *p, "weights")
        check(m, *m1, "exp_avg")
        check(v, *v1, "exp_avg_sq")
