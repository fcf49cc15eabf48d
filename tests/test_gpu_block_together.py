"""A whole block of an image network as it is used: rotary positions, attention,
the joint, the gated layer and the second joint, forward and gradients, against
the definitions in 64 bits; captured in a graph; and the example made of them."""
import math
import os
import sys

import pytest
import torch
import torch.nn.functional as F

import ssim_loss_amd as S
from block_oracle import act_of, pairs_of, seen_by
from gpu_util import say
from train_oracle import U, joint

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

WIDTH, HEADS, KV, DIM, HIDDEN = 96, 4, 2, 24, 160
AXES = (8, 16)


def weights(dtype, seed=0):
    rng = torch.Generator(device="cuda").manual_seed(seed)
    m = lambda a, b: (torch.randn(a, b, generator=rng, device="cuda") * b ** -0.5).to(dtype).requires_grad_(True)
    v = lambda x: (x + 0.1 * torch.randn(WIDTH, generator=rng, device="cuda")).requires_grad_(True)
    return {"qkv": m((HEADS + 2 * KV) * DIM, WIDTH), "out": m(WIDTH, HEADS * DIM), "gate": m(HIDDEN, WIDTH), "up": m(HIDDEN, WIDTH),
            "down": m(WIDTH, HIDDEN), "scale": v(0.5), "post": v(1.0), "pre": v(1.0), "scale2": v(0.5), "post2": v(1.0),
            "pre2": v(1.0)}


def block(x, h, w, positions, lengths):
    whole = F.linear(h, w["qkv"]).unflatten(-1, (HEADS + 2 * KV, DIM))
    q, k = S.rotary(whole[:, :, :HEADS], whole[:, :, HEADS:HEADS + KV], positions, AXES, pairs="halves")
    y = S.attention(q, k, whole[:, :, HEADS + KV:], causal=True, query_lengths=lengths, key_lengths=lengths)
    x, h = S.block_norm(x, F.linear(y.flatten(2), w["out"]), None, w["scale"], w["post"], w["pre"])
    y = S.gated_linear(h, w["gate"], w["up"], act="gelu")
    return S.block_norm(x, F.linear(y, w["down"]), None, w["scale2"], w["post2"], w["pre2"])


def definition(x, h, w, positions, lengths):
    b, n, _ = h.shape
    whole = (h @ w["qkv"].t()).unflatten(-1, (HEADS + 2 * KV, DIM))
    first, second, rate, axis = pairs_of(AXES, "halves")
    angle = (positions.cpu().double()[..., axis] * torch.exp(rate * math.log(10000.0))).unsqueeze(-2)

    def turned(t):
        # (without writing in place: autograd)
        order = torch.argsort(torch.tensor(first + second))
        a, c = t[..., first], t[..., second]
        return torch.cat([a * angle.cos() - c * angle.sin(), c * angle.cos() + a * angle.sin()], -1)[..., order]

    q, k, v = turned(whole[:, :, :HEADS]), turned(whole[:, :, HEADS:HEADS + KV]), whole[:, :, HEADS + KV:]
    k, v = (t.repeat_interleave(HEADS // KV, 2) for t in (k, v))
    s = torch.matmul(q.transpose(1, 2), k.permute(0, 2, 3, 1).contiguous()) * DIM ** -0.5
    seen = torch.stack([seen_by(n, n, True, int(c), int(c)) for c in lengths.tolist()])[:, None]
    p = torch.softmax(torch.where(seen, s, -1e300), -1) * seen
    y = torch.matmul(p, v.transpose(1, 2)).transpose(1, 2).flatten(2)
    x, h = joint(x, y @ w["out"].t(), None, w["scale"], w["post"], w["pre"], 1e-6, "none")
    g, u = h @ w["gate"].t(), h @ w["up"].t()
    return joint(x, (act_of(g, "gelu")[0] * u) @ w["down"].t(), None, w["scale2"], w["post2"], w["pre2"], 1e-6, "none")


def inputs(dtype, n=70, seed=1):
    rng = torch.Generator(device="cuda").manual_seed(seed)
    f = lambda t, std=1.0: (torch.randn(3, n, WIDTH, generator=rng, device="cuda") * std).to(t)
    at = torch.arange(n, device="cuda")
    return (f(torch.float32).requires_grad_(True), f(dtype).requires_grad_(True), torch.stack([at // 9, at % 9], 1).float(),
            torch.tensor([n, 1, n // 2], dtype=torch.int32, device="cuda"), f(torch.float32, 0.1), f(dtype, 0.1))


# What the norm of a result may be off by, relative: of about 30 stages of the block and its gradient each leaves at
# most the roundings of sums of up to 210 terms in fp32 (a quarter of 2 n U in the norm, since they are not all of one
# sign), or two half steps of bf16, and later ones (norms, a softmax) carry what came before at most twice as far.
FACTOR = {torch.float32: 30 * 2 * 210 * U / 2, torch.bfloat16: 30 * 2 * 2 * 2.0 ** -9}


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_a_block_and_its_gradients(dtype):
    x, h, positions, lengths, dx, dh = inputs(dtype)
    w = weights(dtype)
    leaves = [x, h, *w.values()]
    outs = block(x, h, w, positions, lengths)
    grads = torch.autograd.grad(outs, leaves, (dx, dh))
    wide = [t.detach().cpu().double().requires_grad_(True) for t in leaves]
    want = definition(wide[0], wide[1], dict(zip(w, wide[2:])), positions, lengths)
    wanted = torch.autograd.grad(want, wide, (dx.cpu().double(), dh.cpu().double()))
    for name, a, b in zip(("x", "h", "dx", "dh", *w), (*outs, *grads), (*want, *wanted)):
        off = float((a.detach().cpu().double() - b.detach()).norm() / b.detach().norm())
        say(name, off)
        assert off <= FACTOR[dtype], name


def test_a_captured_training_step_of_a_block():
    x, h, positions, lengths, dx, dh = inputs(torch.bfloat16)
    w = weights(torch.bfloat16)
    leaves = [x, h, *w.values()]

    def step():
        outs = block(x, h, w, positions, lengths)
        return [o.detach() for o in outs], torch.autograd.grad(outs, leaves, (dx, dh))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs, grads = step()
    for replay in range(3):
        say("replay", replay)
        new = inputs(torch.bfloat16, seed=30 + replay)
        with torch.no_grad():
            for to, by in zip((x, h, dx, dh), (new[0], new[1], new[4], new[5])):
                to.copy_(by)
            lengths.sub_(1).clamp_(min=0)
        graph.replay()
        torch.cuda.synchronize()
        eager = step()
        assert all(torch.equal(a, b) for a, b in zip(outs, eager[0]))
        assert all(torch.equal(a, b) for a, b in zip(grads, eager[1]))


def test_two_blocks_at_once_on_two_streams():
    made = [(inputs(torch.bfloat16, seed=40 + k), weights(torch.bfloat16, seed=50 + k)) for k in range(2)]

    def step(k):
        (x, h, positions, lengths, dx, dh), w = made[k]
        outs = block(x, h, w, positions, lengths)
        return [o.detach() for o in outs] + list(torch.autograd.grad(outs, [x, h, *w.values()], (dx, dh)))

    want = [step(0), step(1)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for k in range(2):
        with torch.cuda.stream(streams[k]):
            got.append(step(k))
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_the_example_with_attention_runs_and_its_gradients_are_the_definitions():
    import fit_image

    losses, norms = fit_image.fit(steps=3, size=64, width=128, blocks=2, attention=True)
    assert torch.isfinite(losses).all() and torch.isfinite(norms).all()
    with pytest.raises(ValueError):
        fit_image.Net(64, 100, 1, attention=True)

    # one block's network against the same with plain operators in fp32 on the same bf16 weights
    net = fit_image.Net(64, 128, 1, attention=True)
    up = torch.randn(1, 3, 64, 64, generator=torch.Generator(device="cuda").manual_seed(3), device="cuda") * 0.1
    leaves = net.parameters()
    grads = torch.autograd.grad(net(), leaves, up)

    class Plain:
        @staticmethod
        def rotary(q, k, positions, axes):
            first, second, rate, axis = pairs_of(axes, "adjacent")
            angle = (positions.double()[..., axis] * torch.exp(rate.cuda() * math.log(10000.0))).float().unsqueeze(-2)
            order = torch.argsort(torch.tensor(first + second)).cuda()
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

    plain = fit_image.Net(64, 128, 1, attention=True)
    wide = {id(a): b.detach().float().requires_grad_(True) for a, b in zip(plain.parameters(), leaves)}
    plain.blocks = [tuple(wide[id(t)] for t in b) for b in plain.blocks]
    plain.head, plain.code = wide[id(plain.head)], wide[id(plain.code)]

    held, fit_image.S = fit_image.S, Plain
    try:
        h = plain.attend(plain.code, plain.code.bfloat16().float())
        wanted = torch.autograd.grad(plain.image(h), [wide[id(t)] for t in plain.parameters()], up)
    finally:
        fit_image.S = held
    for a, b in zip(grads, wanted):
        off = float((a.float() - b).norm() / b.norm())
        say(tuple(a.shape), off)
        assert off <= FACTOR[torch.bfloat16]
