"""The gated layer's gradients in fp16 where the gradient that arrives is far from
1: dg and du lie between the products in the type, whose numbers end at 65504 and
lose bits below 2^-14."""
import pytest
import torch

import ssim_loss_amd as S
from block_oracle import Gated
from gpu_util import say
from test_gpu_gated_linear import make, run

pytestmark = pytest.mark.gpu
F16 = torch.float16
SIZES = [1e-6, 1e-5, 1e-3, 1.0, 8e3]


def far_apart(name, got, want):
    """Relative to the norm.  dg and du are each off by at most 2^-11 of themselves (2^-12.2
    in the square mean), independently, and a result by as much again: 4e-4 of the norm
    together, of which 2^-10 is allowed; and half of the smallest step, 2^-25, of each result.
    The errors are sums over the same roundings for all results, small ones (sums that happen to
    cancel) among them: those that fit the type by eight of the errors allowed are judged, with
    their number's share of the whole norm as their limit; those past it by as many are infinite."""
    got, want = got.detach().cpu().double(), want.reshape(got.shape)
    margin = 8 * 2.0 ** -10 * want.square().mean().sqrt()
    fits = want.abs() <= 65504 - margin
    off = torch.where(fits, got - want, 0.0).norm()
    limit = (2.0 ** -10 * want.norm() + 2.0 ** -25 * want.numel() ** 0.5) * fits.double().mean().sqrt()
    say(name, float(off), float(limit))
    assert off <= limit, name
    assert torch.isinf(got[want.abs() > 65536 + margin]).all(), name


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("rows,width,hidden", [
    (300, 256, 200), (40, 264, 136), (2000, 264, 520), (730, 36, 34), (90, 33, 65), (2000, 2040, 4080)])
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_gradients_of_all_sizes(rows, width, hidden, size, act):
    t, d_out = make((rows, width), hidden, F16, seed=31)
    d_out = (d_out.float() * (size / 0.1)).clamp(-60000, 60000).half()
    t["x"][1] *= 4
    _, grads = run(t, d_out, act)
    want = Gated(**t, act=act, d_out=d_out)
    for name in ("x", "w_gate", "w_up", "b_gate", "b_up"):
        far_apart(name, grads[name], want.value[name])


def test_a_gradient_that_is_not_finite_leaves_the_others_right():
    """The largest of the numbers that are left sets the range."""
    t, d_out = make((90, 64), 96, F16, seed=32)
    d_out *= 1e-4
    want = Gated(**t, d_out=d_out)
    for bad in (float("inf"), float("nan")):
        broken = d_out.clone()
        broken[2, 5] = bad
        _, grads = run(t, broken)
        rest = [k for k in range(90) if k != 2]
        far_apart("x", grads["x"][rest], want.value["x"][rest])
        assert not torch.isfinite(grads["x"][2]).any() and not torch.isfinite(grads["w_gate"][5]).any()
        others = [k for k in range(96) if k != 5]
        assert torch.isfinite(grads["w_gate"][others]).all() and torch.isfinite(grads["w_up"][others]).all()


def test_the_range_follows_replays_of_a_graph():
    t, d_out = make((70, 64), 96, F16, seed=33)
    t = {k: v.requires_grad_(True) for k, v in t.items()}
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        grads = torch.autograd.grad(S.gated_linear(**t), list(t.values()), d_out)
    for replay, size in enumerate((1e-6, 8e3, 1.0, 1e-4)):
        new = (make((70, 64), 96, F16, seed=40 + replay)[1].float() * (size / 0.1)).clamp(-60000, 60000).half()
        d_out.copy_(new)
        graph.replay()
        torch.cuda.synchronize()
        want = run(t, new)[1]
        assert all(torch.equal(g, w) for g, w in zip(grads, want.values()))


def test_no_gradient_at_all():
    t, d_out = make((70, 64), 96, F16, seed=34)
    _, grads = run(t, torch.zeros_like(d_out))
    assert not any(g.any() for g in grads.values())
