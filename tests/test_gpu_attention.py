"""Attention on the GPU, forward and gradients, against the definition in 64
bits (bounds: block_oracle)."""
import math

import pytest
import torch

import ssim_loss_amd as S
from block_oracle import Attention
from gpu_util import say

pytestmark = pytest.mark.gpu
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
NAMES = ("q", "k", "v")


def make(batch, n, m, heads, kv, dim, dtype, seed=0, std=1.0):
    rng = torch.Generator(device="cuda").manual_seed(seed)
    f = lambda *s, std=std, mean=0.0: (torch.randn(s, generator=rng, device="cuda") * std + mean).to(dtype)
    t = {"q": f(batch, n, heads, dim, std=1.2 * std), "k": f(batch, m, kv, dim), "v": f(batch, m, kv, dim, mean=0.2)}
    return t, f(batch, n, heads, dim, std=0.1)


def lengths(*n):
    return torch.tensor(n, dtype=torch.int32, device="cuda")


def run(t, d_out, leaves=NAMES, **kw):
    t = {k: v.detach().requires_grad_(k in leaves) for k, v in t.items()}
    out = S.attention(t["q"], t["k"], t["v"], **kw)
    grads = torch.autograd.grad(out, [t[k] for k in leaves], d_out)
    return out.detach(), dict(zip(leaves, grads))


def verify(t, d_out, **kw):
    out, grads = run(t, d_out, **kw)
    torch.cuda.synchronize()
    want = Attention(t["q"], t["k"], t["v"], d_out=d_out, **kw)
    assert out.is_contiguous() and out.dtype == t["q"].dtype
    want.check("out", out)
    for k, g in grads.items():
        assert g.dtype == t[k].dtype and g.shape == t[k].shape
        want.check(k, g)
    with torch.no_grad():  # the call without gradients is the same forward
        assert torch.equal(S.attention(t["q"], t["k"], t["v"], **kw), out)
    return out, grads


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("dim", [8, 16, 32, 40, 64, 72, 80, 96, 104, 128])
def test_widths_of_heads(dim, dtype):
    say("attention", dim, dtype)
    verify(*make(2, 70, 90, 3, 3, dim, dtype, seed=dim))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("n,m", [(1, 1), (1, 2), (2, 1), (31, 33), (32, 32), (33, 31), (63, 65), (64, 64), (65, 63),
                                 (127, 129), (128, 128), (129, 127), (257, 257), (300, 5), (5, 300)])
@pytest.mark.parametrize("causal", [False, True])
def test_lengths(n, m, causal, dtype):
    """With causal order and more queries than keys, the first rows see nothing."""
    say("attention", n, m, causal, dtype)
    out, grads = verify(*make(2, n, m, 2, 2, 64, dtype, seed=n + m), causal=causal)
    if causal and n > m:
        assert not out[:, :n - m].any() and not grads["q"][:, :n - m].any()


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("heads,kv", [(4, 2), (6, 2), (5, 1), (8, 8), (24, 3)])
@pytest.mark.parametrize("causal", [False, True])
def test_shared_key_heads(heads, kv, causal, dtype):
    say("attention", heads, kv, causal, dtype)
    verify(*make(1, 50, 77, heads, kv, 64, dtype, seed=heads), causal=causal)
    verify(*make(2, 3, 150, heads, kv, 40, dtype, seed=heads + 1), causal=causal)


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("causal", [False, True])
def test_ragged_lengths(causal, dtype):
    """Sequences of no, one and all tokens, and lengths outside the tensor's."""
    t, d_out = make(8, 90, 90, 4, 2, 64, dtype, seed=3)
    both = lengths(90, 0, 1, 33, 64, 89, 200, -5)
    say("attention ragged", causal, dtype)
    out, grads = verify(t, d_out, causal=causal, query_lengths=both, key_lengths=both)
    assert not out[1].any() and not out[2, 1:].any() and not out[7].any()
    assert not grads["k"][3, 33:].any() and not grads["v"][3, 33:].any() and not grads["q"][3, 33:].any()
    verify(t, d_out, causal=causal, key_lengths=both)
    verify(t, d_out, causal=causal, query_lengths=both)
    verify(t, d_out, causal=causal, query_lengths=lengths(5, 90, 7, 0, 64, 1, 33, 90),
           key_lengths=lengths(90, 5, 8, 64, 0, 33, 1, 90))


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("causal", [False, True])
def test_what_is_behind_a_sequence_is_not_read(bad, causal, dtype):
    t, d_out = make(3, 100, 100, 4, 2, 72, dtype, seed=4)
    n = lengths(37, 100, 64)
    kw = dict(causal=causal, query_lengths=n, key_lengths=n)
    clean = run(t, d_out, **kw)
    for b, length in enumerate(n.tolist()):
        for x in (*t.values(), d_out):
            x[b, length:] = bad
    got = run(t, d_out, **kw)
    assert torch.equal(got[0], clean[0])
    for k in NAMES:
        assert torch.equal(got[1][k], clean[1][k]), k
    # few rows and many keys take another path
    q = t["q"][:, :3].contiguous()
    q[:] = 1.0
    few = S.attention(q, t["k"], t["v"], key_lengths=n)
    assert torch.isfinite(few).all()


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("dim", [32, 64, 80, 128])
@pytest.mark.parametrize("n,m,heads,kv", [(1, 1500, 8, 2), (1, 3000, 4, 4), (4, 700, 8, 1), (7, 999, 4, 1), (2, 5000, 3, 3)])
def test_few_rows_over_many_keys(n, m, heads, kv, dim, dtype):
    """The keys are split over workgroups; sequences end within the parts."""
    say("attention", n, m, heads, kv, dim, dtype)
    t, d_out = make(3, n, m, heads, kv, dim, dtype, seed=m + n)
    verify(t, d_out)
    verify(t, d_out, causal=True, key_lengths=lengths(m, 1, m // 3))
    verify(t, d_out, key_lengths=lengths(0, 129, m - 1))


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
def test_more_rows_with_the_keys_in_parts(dtype):
    t, d_out = make(1, 60, 2100, 2, 1, 64, dtype, seed=5)
    verify(t, d_out)
    verify(t, d_out, causal=True, key_lengths=lengths(1111))


def test_many_pairs_over_the_xcds():
    verify(*make(8, 40, 50, 4, 2, 32, BF16, seed=6), causal=True)
    verify(*make(5, 40, 50, 3, 3, 32, BF16, seed=7), causal=True)


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("dim", [8, 32, 40, 64, 72, 96, 104, 128])
def test_many_pairs_of_short_sequences(dim, dtype):
    """Waves with 32 rows (or keys) of their own: 864 blocks of 32 rows and more."""
    say("attention many", dim, dtype)
    t, d_out = make(16, 70, 90, 18, 18, dim, dtype, seed=dim + 1)
    verify(t, d_out)
    verify(t, d_out, causal=True)
    t, d_out = make(20, 150, 131, 12, 4, dim, dtype, seed=dim + 2)
    n = lengths(*(0, 1, 150, 149, 33, 32, 128, 129, 64, 96) * 2)
    m = lengths(*(5, 131, 131, 0, 131, 64, 1, 33, 32, 96, 131, 20, 128, 130, 129, 3, 131, 90, 31, 0))
    verify(t, d_out, query_lengths=n, key_lengths=m)
    verify(t, d_out, causal=True, query_lengths=n, key_lengths=m)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("n,m,batch,dim", [(257, 130, 32, 128), (130, 257, 32, 104), (513, 300, 12, 128)])
def test_eight_waves(n, m, batch, dim, dtype):
    """1024 blocks of 256 rows or more: of the queries, of the keys, of both."""
    say("attention eight", n, m, dtype)
    t, d_out = make(batch, n, m, 32, 32, dim, dtype, seed=n)
    verify(t, d_out)
    some = lengths(*(range(1, 1 + n, n // batch))[:batch])
    verify(t, d_out, query_lengths=some, key_lengths=lengths(*(range(m, 0, -(m // batch)))[:batch]))


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
def test_strided_inputs(dtype):
    rng = torch.Generator(device="cuda").manual_seed(8)
    whole = torch.randn(2, 66, 8, 64, generator=rng, device="cuda").to(dtype)
    d_out = torch.randn(2, 66, 4, 64, generator=rng, device="cuda").to(dtype)
    views = {"q": whole[:, :, :4], "k": whole[:, :, 4:6], "v": whole[:, :, 6:]}
    verify(views, d_out, causal=True)
    by_heads = {k: v.transpose(1, 2).contiguous().transpose(1, 2) for k, v in views.items()}
    out, grads = verify(by_heads, d_out, causal=True)
    # at odd elements, with gaps, and expanded: copied first
    odd = {k: torch.cat([v.flatten()[:1], v.flatten()])[1:].view(v.shape) for k, v in views.items()}
    got = run(odd, d_out, causal=True)
    assert torch.equal(got[0], out) and all(torch.equal(got[1][k], grads[k]) for k in NAMES)
    gaps = {k: v.repeat_interleave(2, -1)[..., ::2] for k, v in views.items()}
    got = run(gaps, d_out, causal=True)
    assert torch.equal(got[0], out) and all(torch.equal(got[1][k], grads[k]) for k in NAMES)
    one = {"q": views["q"], "k": views["k"][:, :1].expand(2, 66, 2, 64), "v": views["v"][:1].expand(2, 66, 2, 64)}
    verify(one, d_out)
    late = torch.zeros(2 * 66 * 4 * 64 + 1, dtype=dtype, device="cuda")[1:].view(2, 66, 4, 64).copy_(d_out)
    got = run(views, late, causal=True)
    assert all(torch.equal(got[1][k], grads[k]) for k in NAMES)
    turned = d_out.transpose(0, 1).contiguous().transpose(0, 1)
    assert torch.equal(run(views, turned, causal=True)[1]["q"], grads["q"])


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
def test_large_scores_and_other_scales(dtype):
    """Rows of one key's weight, and of far apart scores."""
    t, d_out = make(1, 70, 130, 2, 2, 64, dtype, seed=9, std=3.0)
    verify(t, d_out, scale=1.0)
    verify(t, d_out, scale=1e-3)
    t["q"][0, 5] = 0.0  # all keys the same
    verify(t, d_out)


@pytest.mark.parametrize("scale", [1e-38, 1e-42])
def test_scales_next_to_nothing(scale):
    """Every key that a row sees has the same weight, wherever the row's first one lies."""
    for n, m in ((40, 200), (300, 200)):
        t, _ = make(1, n, m, 2, 2, 64, F32, seed=17)
        out = S.attention(t["q"], t["k"], t["v"], scale=scale, causal=True)
        want = Attention(t["q"], t["k"], t["v"], scale=scale, causal=True)
        want.check("out", out)


def test_a_gradient_with_its_sign_turned():
    t, d_out = make(1, 40, 50, 2, 2, 64, F32, seed=18)
    q = t["q"].requires_grad_()
    out = S.attention(q, t["k"], t["v"])
    a, = torch.autograd.grad(out, q, -d_out, retain_graph=True)
    b, = torch.autograd.grad(out, q, torch._neg_view(d_out))
    assert torch.equal(a, b)


@pytest.mark.parametrize("size", [1e-4, 200.0])
def test_small_and_large_gradients_in_fp16(size):
    t, d_out = make(1, 128, 700, 2, 2, 64, F16, seed=10)
    verify(t, (d_out.float() * size / 0.1).half())


def test_scores_of_minus_infinity():
    t, _ = make(1, 3, 40, 2, 2, 32, F32, seed=11)
    t["q"][0, 1] = 0.0
    t["q"][0, 1, :, 0] = math.inf
    t["k"][..., 0] = -1.0
    out = S.attention(**t)
    assert not out[0, 1].any() and torch.isfinite(out).all()


def test_any_set_of_leaves():
    t, d_out = make(2, 45, 60, 4, 2, 64, BF16, seed=12)
    want = run(t, d_out)[1]
    for leaf in NAMES:
        assert torch.equal(run(t, d_out, leaves=(leaf,))[1][leaf], want[leaf])


@pytest.mark.parametrize("n,m", [(0, 9), (9, 0), (0, 0)])
def test_no_tokens(n, m):
    t, d_out = make(2, n, m, 4, 2, 64, BF16, seed=13)
    out, grads = run(t, d_out)
    assert out.shape == t["q"].shape and not out.any()
    for k in NAMES:
        assert grads[k].shape == t[k].shape and not grads[k].any()
    t, d_out = make(0, 4, 4, 4, 2, 64, BF16)
    out, grads = run(t, d_out)
    assert out.shape == t["q"].shape


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("batch,n", [(2, 1), (2, 40), (30, 300)])
def test_a_row_of_one_key_has_no_gradient(batch, n, dtype):
    """It gives that key all, whatever their product is."""
    t, d_out = make(batch, n, n, 4, 2, 64, dtype, seed=19)
    _, grads = verify(t, d_out, causal=True)
    assert not grads["q"][:, 0].any()
    m = lengths(*(1 for _ in range(batch)))
    _, grads = verify(t, d_out, key_lengths=m)
    assert not grads["q"].any() and not grads["k"].any() and grads["v"][:, 0].any()


def test_the_same_bits_again():
    t, d_out = make(2, 500, 700, 6, 2, 72, F16, seed=14)
    a, b = run(t, d_out, causal=True), run(t, d_out, causal=True)
    assert torch.equal(a[0], b[0]) and all(torch.equal(a[1][k], b[1][k]) for k in NAMES)


def test_gradients_are_differences():
    """The kernels' gradients along a direction against differences of the
    definition in 64 bits, within the gradients' own bounds."""
    t, d_out = make(1, 12, 17, 2, 1, 16, F32, seed=15)
    grads = run(t, d_out, causal=True)[1]
    want = Attention(t["q"], t["k"], t["v"], causal=True, d_out=d_out)
    wide = {k: v.cpu().double() for k, v in t.items()}
    f = lambda v: float((Attention(v["q"], v["k"], v["v"], causal=True).value["out"] * d_out.cpu().double()).sum())
    TINY64 = 1e-5
    rng = torch.Generator().manual_seed(16)
    from train_oracle import TINY
    TINY.setdefault(torch.float64, 0.0)
    for k, v in wide.items():
        along = torch.randn(v.shape, generator=rng, dtype=torch.float64)
        up, down = ({**wide, k: v + s * along} for s in (TINY64, -TINY64))
        slope = (f(up) - f(down)) / (2 * TINY64)
        got = float((grads[k].cpu().double() * along).sum())
        assert abs(got - slope) <= float((want.off[k] * along.abs()).sum()) + 1e-7 * (1 + abs(slope)), k


def test_past_32_bit_offsets():
    """Keys and values of more than 2^32 bytes, of which the last are looked at."""
    m, heads = 1 << 20, 16
    k = torch.zeros(1, m, heads, 128, dtype=BF16, device="cuda")
    v = torch.zeros_like(k)
    rng = torch.Generator(device="cuda").manual_seed(17)
    far = m - 7
    q = torch.randn(1, 1, heads, 128, generator=rng, device="cuda").bfloat16()
    k[0, far] = 40 * q[0, 0]  # all the weight
    v[0, far] = torch.randn(heads, 128, generator=rng, device="cuda").bfloat16()
    say("attention", m)
    out = S.attention(q, k, v)
    assert torch.allclose(out[0, 0].float(), v[0, far].float(), rtol=2 ** -7, atol=1e-3)
    none = S.attention(q, k, v, key_lengths=lengths(far))
    assert none.abs().max() < 1e-6


def test_on_another_stream():
    t, d_out = make(2, 300, 400, 4, 2, 64, BF16, seed=18)
    want = run(t, d_out)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = run(t, d_out)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(want[0], got[0]) and all(torch.equal(want[1][k], got[1][k]) for k in NAMES)


@pytest.mark.parametrize("n,m", [(130, 130), (1, 2000)])
def test_captured_in_a_graph(n, m):
    """Forward and gradients in one graph, replayed on new inputs and lengths."""
    t, d_out = make(2, n, m, 4, 2, 64, BF16, seed=19)
    t = {k: v.requires_grad_(True) for k, v in t.items()}
    kl = lengths(m, m // 2)

    def step():
        out = S.attention(t["q"], t["k"], t["v"], causal=True, key_lengths=kl)
        return out.detach(), torch.autograd.grad(out, list(t.values()), d_out)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, grads = step()
    for replay in range(4):
        say("replay", replay)
        new, new_d = make(2, n, m, 4, 2, 64, BF16, seed=20 + replay)
        with torch.no_grad():
            for k, v in t.items():
                v.copy_(new[k])
            d_out.copy_(new_d)
            kl.copy_(lengths(m - replay, 1 + replay))
        graph.replay()
        torch.cuda.synchronize()
        want = run(new, new_d, causal=True, key_lengths=kl)
        assert torch.equal(out, want[0])
        assert all(torch.equal(g, want[1][k]) for g, k in zip(grads, NAMES))


def test_captured_with_gradients_beside_an_eager_graph_is_refused():
    t, d_out = make(1, 20, 20, 2, 2, 32, F32, seed=25)
    q = t["q"].requires_grad_(True)
    eager = S.attention(q, t["k"], t["v"])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        d_out * 2.0
        with pytest.raises(RuntimeError, match="default stream"):
            S.attention(q, t["k"], t["v"])
    del eager


def test_passes_through_one_graph_and_changed_inputs():
    t, d_out = make(1, 20, 20, 2, 2, 32, F32, seed=26)
    t = {k: v.requires_grad_(True) for k, v in t.items()}
    out = S.attention(**t)
    a = torch.autograd.grad(out, list(t.values()), d_out, retain_graph=True)
    b = torch.autograd.grad(out, list(t.values()), d_out)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    with pytest.raises(RuntimeError, match="second time"):
        torch.autograd.grad(out, list(t.values()), d_out)
    out = S.attention(**t)
    with torch.no_grad():
        t["k"] += 1
    with pytest.raises(RuntimeError, match="modified"):
        out.sum().backward()
    with pytest.raises(RuntimeError, match="create_graph"):
        torch.autograd.grad(S.attention(**t).sum(), t["q"], create_graph=True)


def test_refusals():
    q, k = torch.zeros(2, 3, 4, 16, device="cuda"), torch.zeros(2, 5, 2, 16, device="cuda")
    f = S.attention
    for call in (lambda: f(q[0], k, k), lambda: f(q, k, k[:, :2]), lambda: f(q, k[:1], k[:1]), lambda: f(q[:, :, :3], k, k),
                 lambda: f(q[..., :12], k[..., :12], k[..., :12]), lambda: f(q, k[..., :8], k[..., :8]),
                 lambda: f(q, k, k, scale=0.0), lambda: f(q, k, k, scale=-1.0), lambda: f(q, k, k, scale=math.nan),
                 lambda: f(q, k, k, key_lengths=lengths(1)), lambda: f(q, k, k, query_lengths=lengths(1, 2, 3)),
                 lambda: f(torch.zeros(1, 1, 1, 136, device="cuda"), *[torch.zeros(1, 1, 1, 136, device="cuda")] * 2)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: f(q, k.half(), k.half()), lambda: f(q, k, k.half()), lambda: f(q.double(), k.double(), k.double()),
                 lambda: f(q, k.cpu(), k), lambda: f(q, k, k, key_lengths=lengths(1, 2).long()),
                 lambda: f(q, k, k, key_lengths=lengths(1, 2).cpu())):
        with pytest.raises(TypeError):
            call()
    with pytest.raises(S.TrainError):
        f(q, k, k, scale=1e300)


@pytest.mark.parametrize("n,m", [(45, 60), (300, 280), (700, 900), (0, 30), (30, 0)])
@pytest.mark.parametrize("dtype", [F32, F16, BF16])
def test_any_set_of_leaves_keeps_the_bits(n, m, dtype):
    """Short sequences' gradients are one launch, longer ones' two."""
    t, d_out = make(1, n, m, 4, 2, 40, dtype, seed=27)
    want = run(t, d_out)[1]
    for leaves in (("q",), ("k",), ("v",), ("q", "v"), ("k", "v")):
        got = run(t, d_out, leaves=leaves)[1]
        assert all(torch.equal(got[k], want[k]) for k in leaves), leaves
