"""What looks at operators through torch's dispatcher does not see the training
operators, so calls within it are refused rather than left out of its result
(no GPU needed: these checks come first)."""
import pytest
import torch
import torch.autograd.forward_ad as forward_ad
from torch.fx.experimental.proxy_tensor import make_fx

import ssim_loss_amd as S


def calls(t):
    """Each entry point on the tensor t."""
    one = torch.ones(4)
    opt = S.AdamW.__new__(S.AdamW)
    opt.params = [t]
    opt.exp_avgs, opt.exp_avg_sqs, opt.masters = [one], [one], None
    opt._step, opt.lr, opt.betas, opt.eps = torch.zeros(2, dtype=torch.int64), 1e-3, (0.9, 0.99), 1e-8
    opt.weight_decay, opt.max_norm = 0.0, None
    return {"x": lambda: S.block_norm(t, one), "branch": lambda: S.block_norm(one, t),
            "gate": lambda: S.block_norm(one, one, gate=t), "scale": lambda: S.block_norm(one, one, scale=t),
            "pre_weight": lambda: S.block_norm(one, one, pre_weight=t),
            "clip": lambda: S.clip_grads_([t, one], 1.0), "norm": lambda: S.grad_norm([t]),
            "params": lambda: opt.step([one]), "grads": lambda: opt.step([t])}


@pytest.mark.parametrize("which", calls(torch.ones(4)))
def test_tensors_with_a_forward_mode_tangent_are_refused(which):
    with forward_ad.dual_level():
        dual = forward_ad.make_dual(torch.ones(4), torch.full((4,), 2.0))
        with pytest.raises(NotImplementedError, match="forward-mode"):
            calls(dual)[which]()
        # one without, within the same level, comes to the next check
        with pytest.raises(TypeError, match="GPU tensor"):
            calls(torch.ones(4))[which]()
    with pytest.raises(TypeError, match="GPU tensor"):
        calls(dual)[which]()


@pytest.mark.parametrize("which", ["x", "clip", "norm", "params"])
@pytest.mark.parametrize("trace", [lambda f, x: torch.jit.trace(f, (x,)), lambda f, x: make_fx(f)(x)],
                         ids=["jit", "fx"])
def test_tracers_are_refused(trace, which):
    def traced(t):
        out = t * 2.0
        calls(t)[which]()
        return out

    with pytest.raises(NotImplementedError, match="tracer"):
        trace(traced, torch.ones(4))
    with pytest.raises(TypeError, match="GPU tensor"):
        traced(torch.ones(4))
