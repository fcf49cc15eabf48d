"""Attention at the ends of its range: scales that fp32 does not hold, scores past
fp32, weights far below a row's largest in fp16, more heads than an int counts."""
import math

import pytest
import torch

import ssim_loss_amd as S
from block_oracle import Attention
from gpu_util import say
from test_gpu_attention import lengths, make, run

pytestmark = pytest.mark.gpu
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("scale", [1e-44, 1e-46, 1e-300])
@pytest.mark.parametrize("n,m", [(40, 200), (300, 200), (1, 3000)])
def test_scales_that_fp32_does_not_hold(n, m, scale, dtype):
    """Each key that a row sees has the same weight, masked or not; no gradient reaches the scores."""
    t, d_out = make(2, n, m, 2, 2, 64, dtype, seed=51)
    for kw in (dict(), dict(causal=True), dict(key_lengths=lengths(m - 3, 7))):
        out, grads = run(t, d_out, scale=scale, **kw)
        want = Attention(t["q"], t["k"], t["v"], scale=scale, d_out=d_out, **kw)
        want.check("out", out)
        for name in ("q", "k", "v"):
            want.check(name, grads[name])


@pytest.mark.parametrize("n", [40, 300, 5000])
@pytest.mark.parametrize("scale", [1e-43, 1e-46])
def test_gradients_with_a_scale_that_fp32_holds_in_few_bits(n, scale):
    """Keys of 10^30 bring the queries' gradient back to numbers that fp32 holds."""
    t, d_out = make(1, n, 90, 2, 1, 64, F32, seed=52)
    t["k"] *= 1e30
    _, grads = run(t, d_out, scale=scale)
    want = Attention(t["q"], t["k"], t["v"], scale=scale, d_out=d_out)
    assert want.value["q"].abs().max() > 1e-20
    want.check("q", grads["q"])


SHAPES = [(40, 200), (300, 200), (1, 3000), (9000, 130)]  # rows shared by waves, keys in parts, rows of a wave's own


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("n,m", SHAPES)
def test_scores_past_fp32_are_not_taken_for_rows_without_keys(n, m, dtype):
    t, _ = make(1, n, m, 2, 2, 64, dtype, seed=53)
    t["q"][:] = t["q"][:, :1].clone()
    t["k"][:, 5] = 8 * t["q"][:, 0].sign()  # the largest score by far
    for scale in (3e37, 1e30, 1e8):
        assert torch.isnan(S.attention(t["q"], t["k"], t["v"], scale=scale)).all(), scale
    for scale in (4e4, 1e3):
        # that key has it all: its weight is rounded to a half type, the product with 1 / sum three
        # times, the result once
        out, want = S.attention(t["q"], t["k"], t["v"], scale=scale).double(), t["v"][:, 5:6].double()
        step = 0.0 if dtype == F32 else torch.finfo(dtype).eps / 2
        assert ((out - want).abs() <= want.abs() * (2.01 * step + 4 * 2.0 ** -24) + 2.0 ** -25).all(), scale


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("n,m", SHAPES)
@pytest.mark.parametrize("low", [-1e8, -1e12, -1e30, -3e38])
def test_keys_far_below_the_others(low, n, m, dtype):
    """They come first, and with the others they have no weight; rows that see no others give zeros."""
    t, _ = make(1, n, m, 2, 2, 64, dtype, seed=54)
    t["q"][..., 0] = 1.0
    t["k"][..., 0] = 0.0
    t["k"][:, :100, :, 1:] = 0.0
    t["k"][:, :100, :, 0] = low
    out = S.attention(t["q"], t["k"], t["v"])
    want = Attention(t["q"], t["k"][:, 100:], t["v"][:, 100:])
    want.check("out", out)
    if low < -1e11:
        assert not S.attention(t["q"], t["k"], t["v"], key_lengths=lengths(100)).any()


@pytest.mark.parametrize("n", [1, 40])
def test_weights_far_below_a_rows_largest_in_fp16(n):
    """2^17 keys of 2^-26 of the largest weight each are 2^-9 of the result.  A weight,
    rounded times 2^7 at least, is off by 2^-25 2^-7 = 2^-32 at most; a result by half a
    step; the sums of positive terms by 2 m U of themselves."""
    m, heads, dim = 1 << 17, 520, 32  # (heads enough that no keys are in parts, whose largest weights would differ)
    k = torch.zeros(1, m, 1, dim, dtype=F16, device="cuda")
    k[:, 0, :, 0] = 18.0
    v = torch.ones(1, m, 1, dim, dtype=F16, device="cuda")
    v[:, 0] = 0.0
    q = torch.zeros(1, n, heads, dim, dtype=F16, device="cuda")
    q[..., 0] = 1.0
    say("attention", n, m)
    out = S.attention(q, k.expand(1, m, heads, dim), v.expand(1, m, heads, dim), scale=1.0)
    w = (m - 1) * math.exp(-18.0)
    want = w / (1 + w)
    off = float((out.double() - want).abs().max())
    assert off <= m * 2.0 ** -32 + want * (2.0 ** -11 + 1e-5), (off, want)


def test_more_heads_than_an_int_counts():
    one = torch.zeros(1, 1, 1, 8, dtype=F16, device="cuda")
    many = one.expand(1, 1, (1 << 32) + 1, 8)
    position = torch.zeros(1, 1, device="cuda")
    for call in (lambda: S.attention(many, one, one), lambda: S.attention(many, many, many),
                 lambda: S.rotary(many, None, position, (8,)), lambda: S.rotary(one, many, position, (8,))):
        with pytest.raises(ValueError, match="heads"):
            call()


@pytest.mark.parametrize("dtype,most", [(F32, 2.0 ** 31), (F16, 2.0 ** 28), (BF16, 2.0 ** 31), (F16, 2.0 ** 23), (F16, 2.0 ** 24)])
@pytest.mark.parametrize("n,m", SHAPES)
def test_scores_up_to_the_bound_stay_numbers(n, m, dtype, most):
    """Keys one after the other a little above those before, up to the largest score that is
    taken: no probability passes the type, none of the row's keys is lost.  The largest differ
    by less than fp32 tells apart, so the weights between them are free."""
    dim = 8
    steps = torch.linspace(0.97, 0.999, m, device="cuda", dtype=torch.float64)
    for way in (steps, steps.flip(0), steps[torch.randperm(m, generator=torch.Generator().manual_seed(1)).cuda()]):
        q, k = torch.zeros(1, n, 2, dim, device="cuda", dtype=dtype), torch.zeros(1, m, 2, dim, device="cuda", dtype=dtype)
        q[..., 0], q[..., 1] = 1.0, 1.0
        k[..., 0] = (way * 1024).to(dtype)[None, :, None]  # (a score is a sum of two, to tell more apart in a half type)
        k[..., 1] = (way * 1024 - k[0, :, 0, 0].double()).to(dtype)[None, :, None]
        out = S.attention(q, k, torch.ones_like(k), scale=most / 1.4427 / 1024)
        assert ((out.double() - 1).abs() < 0.02).all()
