"""Rotary positions with several axes on the GPU against the definition in 64
bits (bounds: block_oracle)."""
import math

import pytest
import torch

import ssim_loss_amd as S
from block_oracle import check, rotary
from gpu_util import say

pytestmark = pytest.mark.gpu
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


def normal(*shape, dtype=F32, seed=0, offset=0):
    rng = torch.Generator(device="cuda").manual_seed(seed)
    n = math.prod(shape)
    return torch.randn(n + offset, generator=rng, device="cuda").to(dtype)[offset:].view(shape)


def grid(tokens, axes, side=7):
    t = torch.arange(tokens, device="cuda")
    return torch.stack([t // side ** (axes - 1 - a) % side if a else t // side ** (axes - 1) for a in range(axes)], 1)


def verify(q, k, positions, axes, base=10000.0, pairs="adjacent"):
    q, k = q.detach().requires_grad_(True), None if k is None else k.detach().requires_grad_(True)
    out = S.rotary(q, k, positions, axes, base=base, pairs=pairs)
    assert out[1] is None if k is None else out[1].dtype == k.dtype
    for x, y, name in ((q, out[0], "q"), (k, out[1], "k")):
        if x is None:
            continue
        assert y.is_contiguous() and y.dtype == x.dtype
        check(y, *rotary(x, positions, axes, base, pairs), name)
        up = normal(*x.shape, dtype=x.dtype, seed=91)
        (grad,) = torch.autograd.grad(y, x, up, retain_graph=True)
        check(grad, *rotary(up, positions, axes, base, pairs, -1.0), "gradient of " + name)
    with torch.no_grad():
        again = S.rotary(q, k, positions, axes, base=base, pairs=pairs)
    assert torch.equal(again[0], out[0]) and (k is None or torch.equal(again[1], out[1]))
    return out


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("pairs", ["adjacent", "halves"])
@pytest.mark.parametrize("dim,axes", [
    (128, (32, 48, 48)), (72, (32, 32)), (64, (64,)), (64, (16, 24, 24)), (80, (26, 26, 26)), (2, (2,)), (7, (2, 4)),
    (40, (6, 10)), (96, (24, 24, 24, 24)), (512, (512,)), (512, (128, 130, 126)), (33, (16, 16)), (20, (8, 8)), (12, (8,))])
def test_heads_and_axes(dim, axes, pairs, dtype):
    say("rotary", dim, axes, pairs, dtype)
    verify(normal(2, 37, 5, dim, dtype=dtype, seed=1), normal(2, 37, 2, dim, dtype=dtype, seed=2),
           grid(37, len(axes)).float(), axes, pairs=pairs)


@pytest.mark.parametrize("shape", [(1, 1, 1), (1, 1, 32), (3, 1, 7), (1, 1000, 1), (2, 333, 16), (70, 3, 2)])
def test_shapes(shape):
    b, t, h = shape
    say("rotary", shape)
    verify(normal(b, t, h, 64, dtype=BF16, seed=3), None, grid(t, 2), (32, 32))


@pytest.mark.parametrize("kind", [torch.float32, torch.int32, torch.int64])
def test_positions_of_each_type_and_of_each_sample(kind):
    rng = torch.Generator(device="cuda").manual_seed(4)
    p = torch.randint(-3000, 100000, (3, 11, 3), generator=rng, device="cuda").to(kind)
    verify(normal(3, 11, 4, 96, seed=5), normal(3, 11, 4, 96, seed=6), p, (32, 32, 32), pairs="halves")
    one = p[:1]
    verify(normal(3, 11, 4, 96, seed=5), None, one.expand(3, 11, 3), (32, 32, 32))
    verify(normal(3, 11, 4, 96, seed=5), None, one, (32, 32, 32))
    verify(normal(3, 11, 4, 96, seed=5), None, p.flip(2).transpose(0, 1).contiguous().transpose(0, 1), (32, 32, 32))


def test_far_and_fractional_positions_keep_their_angle():
    p = torch.tensor([[0.0], [0.25], [1e5 + 0.5], [-1e6], [2.0 ** 31], [3e7]], device="cuda")
    verify(normal(1, 6, 2, 64, seed=7), None, p, (64,))
    verify(normal(1, 6, 2, 64, seed=7), None, p, (64,), base=1.5)
    far = torch.tensor([[2 ** 40 + 1], [-(2 ** 40) - 3]], device="cuda")
    verify(normal(1, 2, 2, 64, seed=8), None, far, (64,))


def test_views_of_one_projection_and_odd_starts():
    whole = normal(2, 19, 9, 64, dtype=BF16, seed=9)
    verify(whole[:, :, :4], whole[:, :, 4:6], grid(19, 2), (32, 32))
    by_heads = normal(2, 4, 19, 64, dtype=BF16, seed=10).transpose(1, 2)
    verify(by_heads, None, grid(19, 2), (32, 32))
    verify(normal(2, 19, 3, 64, dtype=F16, seed=11, offset=1), None, grid(19, 2), (32, 32), pairs="halves")
    apart = normal(2, 19, 3, 64, 2, dtype=F32, seed=12)[..., 0]  # the last dimension strided
    verify(apart, None, grid(19, 2), (32, 32))
    verify(normal(1, 19, 3, 64, seed=13).expand(4, 19, 3, 64), None, grid(19, 2), (32, 32))


def test_elements_behind_the_axes_pass_as_they_are():
    q = normal(1, 5, 3, 40, dtype=F16, seed=14)
    q[0, 2, 1, 33] = math.nan
    q[0, 3, 1, 34] = math.inf
    y, _ = S.rotary(q, None, grid(5, 1), (32,))
    assert torch.equal(y[..., 32:].view(torch.int16), q[..., 32:].view(torch.int16))


def test_a_token_that_is_not_finite_stays_alone():
    q = normal(1, 6, 3, 32, seed=15)
    p = grid(6, 1).float()
    clean, _ = S.rotary(q, None, p, (32,))
    p[2] = math.nan
    p[4] = math.inf
    y, _ = S.rotary(q, None, p, (32,))
    rest = [0, 1, 3, 5]
    assert torch.equal(y[:, rest], clean[:, rest]) and torch.isnan(y[:, [2, 4]]).all()


@pytest.mark.parametrize("shape", [(0, 4, 2), (2, 0, 2)])
def test_nothing_to_turn(shape):
    q = normal(*shape, 32).requires_grad_(True)
    y, _ = S.rotary(q, None, torch.zeros(shape[1], 1, device="cuda"), (32,))
    assert y.shape == q.shape
    (g,) = torch.autograd.grad(y.sum(), q)
    assert g.shape == q.shape


def test_one_of_two_gradients():
    q, k = normal(1, 9, 4, 32, seed=16).requires_grad_(True), normal(1, 9, 2, 32, seed=17).requires_grad_(True)
    p = grid(9, 1)
    a, b = S.rotary(q, k, p, (32,))
    up = normal(1, 9, 2, 32, seed=18)
    (gk,) = torch.autograd.grad(b, k, up)
    check(gk, *rotary(up, p, (32,), 10000.0, "adjacent", -1.0), "k")
    gq = torch.autograd.grad(S.rotary(q, k.detach(), p, (32,))[0].sum(), q)[0]
    check(gq, *rotary(torch.ones_like(q), p, (32,), 10000.0, "adjacent", -1.0), "q")


def test_past_32_bit_offsets():
    tokens = (1 << 31) // (64 * 512) + 5
    q = torch.zeros(1, tokens, 64, 512, dtype=BF16, device="cuda")
    some = [0, tokens // 2, tokens - 1]
    for k in some:
        q[:, k] = normal(64, 512, dtype=BF16, seed=k)
    p = torch.arange(tokens, device="cuda")[:, None]
    say("rotary", tuple(q.shape))
    y, _ = S.rotary(q, None, p, (512,), pairs="halves")
    check(y[:, some], *rotary(q[:, some], p[some], (512,), 10000.0, "halves"), "far rows")


def test_on_another_stream_and_captured():
    q, k, p = normal(2, 40, 4, 64, dtype=BF16, seed=19), normal(2, 40, 2, 64, dtype=BF16, seed=20), grid(40, 2).float()
    want = S.rotary(q, k, p, (32, 32))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = S.rotary(q, k, p, (32, 32))
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, z = S.rotary(q, k, p, (32, 32))
    for replay in range(3):
        q.copy_(normal(2, 40, 4, 64, dtype=BF16, seed=30 + replay))
        p.add_(1.0)
        graph.replay()
        torch.cuda.synchronize()
        want = S.rotary(q, k, p, (32, 32))
        assert torch.equal(y, want[0]) and torch.equal(z, want[1])


def test_refusals():
    q, p = torch.zeros(2, 3, 4, 8, device="cuda"), torch.zeros(3, 1, device="cuda")
    f = S.rotary
    for call in (lambda: f(q[0], None, p, (8,)), lambda: f(q, q[:1], p, (8,)), lambda: f(q, q[:, :2], p, (8,)),
                 lambda: f(q, q[..., :4], p, (8,)), lambda: f(q[:, :, :0], q, p, (8,)), lambda: f(q, q[:, :, :0], p, (8,)), lambda: f(q, None, p, (7,)), lambda: f(q, None, p, (10,)),
                 lambda: f(q, None, p, (0,)), lambda: f(q, None, p, ()), lambda: f(q, None, p, (4, 4)),
                 lambda: f(q, None, torch.zeros(3, 2, device="cuda"), (6, 4)),
                 lambda: f(q, None, torch.zeros(2, 1, device="cuda"), (8,)),
                 lambda: f(q, None, torch.zeros(3, 3, 1, device="cuda"), (8,)),
                 lambda: f(q, None, p[:, 0], (8,)), lambda: f(q, None, p, (8,), base=0.0),
                 lambda: f(q, None, p, (8,), base=math.nan), lambda: f(q, None, p, (8,), pairs="both"),
                 lambda: f(torch.zeros(1, 1, 1, 514, device="cuda"), None, torch.zeros(1, 1, device="cuda"), (514,))):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: f(q, q.half(), p, (8,)), lambda: f(q, None, p.cpu(), (8,)), lambda: f(q, None, p.half(), (8,)),
                 lambda: f(q.double(), None, p, (8,)), lambda: f(q, q.cpu(), p, (8,)), lambda: f(q.cpu(), None, p, (8,))):
        with pytest.raises(TypeError):
            call()
    with pytest.raises(NotImplementedError, match="positions"):
        f(q, None, p.clone().requires_grad_(True), (8,))
    a = q.clone().requires_grad_(True)
    with pytest.raises(RuntimeError, match="create_graph"):
        torch.autograd.grad(f(a, None, p, (8,))[0].sum(), a, create_graph=True)
