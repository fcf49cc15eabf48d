"""How near the operators inside a block come to the definition in 64 bits, by the
norm of a whole result.  The bounds of block_oracle hold for every element whatever
the signs of the roundings; these limits count roundings as independent, and notice
a term that is a hundredth off.

A rounding to a type is off by EPS of the value in the square mean: a step over
sqrt(12), where a value lies anywhere in its binade (2^-7 sqrt(0.541 / 12) in bf16)."""
import math
import os
import sys

import pytest
import torch
import torch.nn.functional as F

import ssim_loss_amd as S
import test_gpu_block_together as together
from block_oracle import Attention, Gated, pairs_of
from gpu_util import say
from test_gpu_attention import lengths, make as make_attention, run as run_attention
from test_gpu_gated_linear import make as make_gated, run as run_gated
from train_oracle import U, joint

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
EPS = {F16: 2.0 ** -10 * math.sqrt(0.541 / 12), BF16: 2.0 ** -7 * math.sqrt(0.541 / 12)}
# Two roundings on the way to each result: of the operand that lies between the products, and its own.  Half as
# much again is allowed.  fp32: some sums of up to some hundred terms, each off by U of the largest part sum.
LIMIT = {F32: 64 * U, F16: 1.5 * math.sqrt(2) * EPS[F16], BF16: 1.5 * math.sqrt(2) * EPS[BF16]}


def near(name, got, want, limit):
    want = want.reshape(got.shape)
    off = float((got.detach().cpu().double() - want).norm() / want.norm())
    say(name, f"{off:.3e} of {limit:.3e}")
    assert off <= limit, name


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("batch,n,m,heads,kv,dim,causal", [
    (2, 70, 90, 3, 3, 64, False), (2, 200, 200, 4, 2, 128, True), (1, 60, 2100, 2, 1, 64, False), (1, 1, 3000, 4, 4, 128, False),
    (16, 130, 140, 18, 18, 72, True), (1, 700, 20, 8, 8, 32, False)])
def test_attention(batch, n, m, heads, kv, dim, causal, dtype):
    t, d_out = make_attention(batch, n, m, heads, kv, dim, dtype, seed=61)
    out, grads = run_attention(t, d_out, causal=causal)
    want = Attention(t["q"], t["k"], t["v"], causal=causal, d_out=d_out).value
    near("out", out, want["out"], LIMIT[dtype])
    for name in ("q", "k", "v"):
        near(name, grads[name], want[name], LIMIT[dtype])


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("n,batch", [(33, 1), (300, 1), (150, 40)])
def test_values_far_larger_than_their_differences(n, batch, dtype):
    """delta_i = do_i . o_i and do_i . v_j are both some size / std = 100 times their difference
    (do_i . (v_j - o_i), with values of the standard deviation std about their mean), so that o's
    rounding to the type, 100 EPS of that, may not come into delta.  What remains: 100 roundings of
    probabilities, which average out over m keys."""
    m, size, std = 1024, 30.0, 0.3
    t, d_out = make_attention(batch, n, m, 2, 2, 64, dtype, seed=62, std=std)
    t["v"] = (t["v"].float() - 0.2 + size).to(dtype)
    _, grads = run_attention(t, d_out)
    want = Attention(t["q"], t["k"], t["v"], d_out=d_out).value
    limit = 1.5 * math.sqrt(2 + (size / std) ** 2 / m) * EPS[dtype]
    near("q", grads["q"], want["q"], limit)
    near("k", grads["k"], want["k"], limit)


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("rows,width,hidden", [(5, 200, 300), (300, 256, 200), (2000, 264, 520), (90, 33, 65)])
@pytest.mark.parametrize("act", ["silu", "gelu", "sigmoid"])
def test_gated_layer(rows, width, hidden, act, dtype):
    t, d_out = make_gated((rows, width), hidden, dtype, seed=63)
    out, grads = run_gated(t, d_out, act)
    want = Gated(**t, act=act, d_out=d_out).value
    near("out", out, want["out"], LIMIT[dtype])
    for name, g in grads.items():
        near(name, g, want[name], LIMIT[dtype])


# Of some 30 stages of a block and its gradient each leaves two roundings of its own, and what is later in the way (norms,
# a softmax) carries what came before at most twice as far: independently, sqrt(30) 2 sqrt(2) EPS.  fp32: 28 U a stage
# (sums of up to 800 terms), which are added as they are.
BLOCK = {F32: 30 * 2 * 28 * U, BF16: math.sqrt(30) * 2 * math.sqrt(2) * EPS[BF16]}


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_a_block(dtype):
    x, h, positions, ends, dx, dh = together.inputs(dtype, seed=64)
    w = together.weights(dtype, seed=65)
    leaves = [x, h, *w.values()]
    outs = together.block(x, h, w, positions, ends)
    grads = torch.autograd.grad(outs, leaves, (dx, dh))
    wide = [t.detach().cpu().double().requires_grad_(True) for t in leaves]
    want = together.definition(wide[0], wide[1], dict(zip(w, wide[2:])), positions, ends)
    wanted = torch.autograd.grad(want, wide, (dx.cpu().double(), dh.cpu().double()))
    for name, a, b in zip(("x", "h", "dx", "dh", *w), (*outs, *grads), (*want, *wanted)):
        near(name, a, b.detach(), BLOCK[dtype])


class Plain:
    """The operators' definitions as torch's own, in 64 bits on the CPU."""

    @staticmethod
    def rotary(q, k, positions, axes):
        first, second, rate, axis = pairs_of(axes, "adjacent")
        angle = (positions.cpu().double()[..., axis] * torch.exp(rate * math.log(10000.0))).unsqueeze(-2)
        order = torch.argsort(torch.tensor(first + second))
        f = lambda t: torch.cat([t[..., first] * angle.cos() - t[..., second] * angle.sin(),
                                 t[..., second] * angle.cos() + t[..., first] * angle.sin()], -1)[..., order]
        return f(q), f(k)

    @staticmethod
    def attention(q, k, v):
        s = torch.matmul(q.transpose(1, 2), k.permute(0, 2, 3, 1).contiguous()) * q.shape[-1] ** -0.5
        return torch.matmul(torch.softmax(s, -1), v.transpose(1, 2).contiguous()).transpose(1, 2)

    @staticmethod
    def gated_linear(x, w_gate, w_up):
        g = F.linear(x, w_gate)
        return g * torch.sigmoid(g) * F.linear(x, w_up)

    @staticmethod
    def block_norm(x, branch, gate, scale, post, pre):
        return joint(x, branch, gate, scale, post, pre, 1e-6, "none")


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_the_example_with_attention(dtype):
    """One block of its network, with the weights in each type, against the definitions."""
    import fit_image

    net = fit_image.Net(64, 128, 1, attention=True)
    leaves = net.parameters()
    up = torch.randn(1, 3, 64, 64, generator=torch.Generator(device="cuda").manual_seed(3), device="cuda") * 0.1

    def with_weights(make):
        made = {id(t): make(t.detach()).requires_grad_(True) for t in leaves}
        other = fit_image.Net(64, 128, 1, attention=True)
        other.blocks = [tuple(made[id(t)] for t in b) for b in net.blocks]
        other.head, other.code = made[id(net.head)], made[id(net.code)]
        return other, [made[id(t)] for t in leaves]

    if dtype == BF16:
        grads = torch.autograd.grad(net(), leaves, up)
    else:
        wide, own = with_weights(lambda t: t.float())
        grads = torch.autograd.grad(wide.image(wide.attend(wide.code, wide.code)), own, up)
    plain, held = with_weights(lambda t: t.cpu().double())
    start = plain.code.bfloat16().double() if dtype == BF16 else plain.code
    kept, fit_image.S = fit_image.S, Plain
    try:
        h = plain.attend(plain.code, start)
        n = plain.side // fit_image.PATCH
        # (image() goes by fp32)
        pixels = torch.sigmoid(F.linear(h, plain.head)).view(n, n, 3, fit_image.PATCH, fit_image.PATCH)
        image = pixels.permute(2, 0, 3, 1, 4).reshape(1, 3, plain.side, plain.side)
        wanted = torch.autograd.grad(image, held, up.cpu().double())
    finally:
        fit_image.S = kept
    for a, b in zip(grads, wanted):
        near(tuple(a.shape), a, b, BLOCK[dtype])
