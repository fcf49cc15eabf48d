"""The gated layer on the GPU, forward and gradients, against the definition in
64 bits (bounds: block_oracle)."""
import math

import pytest
import torch

import ssim_loss_amd as S
from block_oracle import Gated
from gpu_util import say

pytestmark = pytest.mark.gpu
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
NAMES = ("x", "w_gate", "w_up", "b_gate", "b_up")


def make(shape, hidden, dtype, bias=True, seed=0, offset=0):
    rng = torch.Generator(device="cuda").manual_seed(seed)

    def f(*s, std=1.0):
        flat = (torch.randn(math.prod(s) + offset, generator=rng, device="cuda") * std).to(dtype)
        return flat[offset:].view(s)

    width = shape[-1]
    t = {"x": f(*shape), "w_gate": f(hidden, width, std=1.5 * width ** -0.5), "w_up": f(hidden, width, std=width ** -0.5)}
    if bias:
        t.update(b_gate=f(hidden, std=0.3), b_up=f(hidden, std=0.3))
    return t, f(*shape[:-1], hidden, std=0.1)


def run(t, d_out, act="silu", leaves=NAMES):
    leaves = [k for k in leaves if k in t]
    t = {k: v.detach().requires_grad_(k in leaves) for k, v in t.items()}
    out = S.gated_linear(**t, act=act)
    return out.detach(), dict(zip(leaves, torch.autograd.grad(out, [t[k] for k in leaves], d_out)))


def verify(t, d_out, act="silu"):
    out, grads = run(t, d_out, act)
    torch.cuda.synchronize()
    want = Gated(**t, act=act, d_out=d_out)
    assert out.dtype == t["x"].dtype
    want.check("out", out)
    for k, g in grads.items():
        assert g.dtype == t[k].dtype and g.shape == t[k].shape
        want.check(k, g)
    with torch.no_grad():
        assert torch.equal(S.gated_linear(**t, act=act), out)
    return out, grads


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("rows,width,hidden", [
    (1, 64, 64), (3, 200, 100), (16, 128, 48), (17, 128, 48), (33, 256, 130), (64, 512, 96), (65, 64, 64), (100, 72, 40),
    (128, 128, 128), (129, 136, 129), (257, 384, 256), (300, 33, 65), (70, 7, 9), (5, 3, 11), (90, 1, 1), (1, 1, 1),
    (514, 384, 1024), (200, 1153, 299), (2, 1153, 301), (1, 8, 17), (66, 1000, 1001)])
def test_shapes(rows, width, hidden, dtype):
    say("gated", rows, width, hidden, dtype)
    verify(*make((rows, width), hidden, dtype, seed=rows + width))


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("act", ["silu", "gelu", "sigmoid"])
@pytest.mark.parametrize("bias", [False, True])
def test_activations(act, bias, dtype):
    verify(*make((2, 45, 96), 160, dtype, bias=bias, seed=3), act=act)
    verify(*make((9, 96), 160, dtype, bias=bias, seed=4), act=act)


def test_one_bias():
    t, d_out = make((80, 64), 72, BF16, seed=5)
    for gone in ("b_gate", "b_up"):
        some = {k: v for k, v in t.items() if k != gone}
        out, grads = run(some, d_out)
        want = Gated(**some, d_out=d_out)
        want.check("out", out)
        for k in grads:
            want.check(k, grads[k])


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("rows,width,hidden", [(2000, 264, 520), (700, 520, 2056), (3000, 136, 72)])
def test_tiles_of_both_sizes(rows, width, hidden, dtype):
    say("gated", rows, width, hidden, dtype)
    verify(*make((rows, width), hidden, dtype, seed=6))


@pytest.mark.parametrize("dtype", [F16, F32])
def test_the_large_tiles(dtype):
    """Enough tiles of 256 x 256 for every CU, the last ones cut."""
    say("gated large", dtype)
    verify(*make((4100, 1032), 2056, dtype, bias=False, seed=7))


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("rows,width,hidden", [(4090, 264, 2040), (4090, 4000, 72), (264, 2040, 4080), (2000, 2040, 4080)])
def test_the_large_tiles_of_each_product(rows, width, hidden, dtype):
    """256 tiles of 256 x 256, one to a CU: of the forward, of the gradient of x, of the
    weights', of both the first and the last."""
    say("gated large", rows, width, hidden, dtype)
    verify(*make((rows, width), hidden, dtype, seed=16))


@pytest.mark.parametrize("rows,width,hidden,dtype", [
    (145, 34, 438, BF16), (132, 35, 115, F32), (730, 36, 34, F16), (233, 35, 32, F32), (3270, 67, 2248, F32),
    (8651, 785, 66, F32), (36639, 2095, 69, BF16), (135, 4249, 6778, F32), (5774, 145, 4180, F32)])
def test_the_summed_axis_in_parts(rows, width, hidden, dtype):
    """Of the gradient of x or the weights', with each size of tile."""
    say("gated parts", rows, width, hidden, dtype)
    verify(*make((rows, width), hidden, dtype, seed=17))


@pytest.mark.parametrize("rows", [3, 80])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_tensors_that_start_anywhere(rows, dtype):
    verify(*make((rows, 128), 72, dtype, seed=8, offset=1))
    verify(*make((rows, 99), 75, dtype, seed=9, offset=3))


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
def test_gates_at_the_ends(dtype):
    t, d_out = make((70, 64), 64, dtype, seed=10)
    t["b_gate"][0::3] = 60.0
    t["b_gate"][1::3] = -60.0
    for act in ("silu", "gelu", "sigmoid"):
        out, grads = verify(t, d_out, act)
        assert all(torch.isfinite(g).all() for g in (out, *grads.values()))


@pytest.mark.parametrize("rows", [5, 90])
def test_a_row_that_is_not_finite_stays_alone(rows):
    t, d_out = make((rows, 100), 130, BF16, seed=11)
    clean = run(t, d_out)
    t["x"][2, 99] = math.nan
    out, grads = run(t, d_out)
    rest = [k for k in range(rows) if k != 2]
    assert torch.equal(out[rest], clean[0][rest]) and torch.isnan(out[2]).all()
    assert torch.equal(grads["x"][rest], clean[1]["x"][rest])


def test_any_set_of_leaves():
    t, d_out = make((70, 64), 96, F16, seed=12)
    want = run(t, d_out)[1]
    for leaf in NAMES:
        assert torch.equal(run(t, d_out, leaves=(leaf,))[1][leaf], want[leaf]), leaf


@pytest.mark.parametrize("shape", [(0, 32), (3, 0, 32)])
def test_no_rows(shape):
    t, d_out = make(shape, 48, F32, seed=13)
    out, grads = run(t, d_out)
    assert out.shape == (*shape[:-1], 48)
    for k, g in grads.items():
        assert g.shape == t[k].shape and not g.any()


def test_upstream_gradients_that_are_not_contiguous():
    t, d_out = make((6, 12, 64), 40, F32, seed=14)
    want = run(t, d_out)[1]
    got = run(t, d_out.transpose(0, 1).contiguous().transpose(0, 1))[1]
    assert all(torch.equal(got[k], want[k]) for k in want)


def test_the_same_bits_again():
    t, d_out = make((1000, 200), 300, BF16, seed=15)
    a, b = run(t, d_out), run(t, d_out)
    assert torch.equal(a[0], b[0]) and all(torch.equal(a[1][k], b[1][k]) for k in a[1])


@pytest.mark.parametrize("act", ["silu", "gelu", "sigmoid"])
def test_gradients_are_differences(act):
    t, d_out = make((5, 12), 9, F32, seed=16)
    grads = run(t, d_out, act)[1]
    want = Gated(**t, act=act, d_out=d_out)
    wide = {k: v.cpu().double() for k, v in t.items()}
    from train_oracle import TINY
    TINY.setdefault(torch.float64, 0.0)
    f = lambda v: float((Gated(**v, act=act).value["out"] * d_out.cpu().double()).sum())
    rng = torch.Generator().manual_seed(17)
    step = 1e-5
    for k, v in wide.items():
        along = torch.randn(v.shape, generator=rng, dtype=torch.float64)
        up, down = ({**wide, k: v + s * along} for s in (step, -step))
        slope = (f(up) - f(down)) / (2 * step)
        got = float((grads[k].cpu().double() * along).sum())
        assert abs(got - slope) <= float((want.off[k] * along.abs()).sum()) + 1e-7 * (1 + abs(slope)), k


def test_past_32_bit_offsets():
    rows, width = (1 << 31) // 1024 + 3, 1024
    x = torch.zeros(rows, width, dtype=BF16, device="cuda")
    some = [0, rows // 2, rows - 1]
    t, _ = make((3, width), 40, BF16, seed=18)
    for at, k in enumerate(some):
        x[k] = t["x"][at]
    say("gated", rows, width)
    out = S.gated_linear(x, t["w_gate"], t["w_up"])
    want = Gated(t["x"], t["w_gate"], t["w_up"])
    want.check("out", out[some])
    assert int(out.count_nonzero(1).ne(0).sum()) == 3


@pytest.mark.parametrize("rows", [7, 300])
def test_streams_and_graphs(rows):
    t, d_out = make((rows, 96), 136, BF16, seed=19)
    want = run(t, d_out)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = run(t, d_out)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(want[0], got[0]) and all(torch.equal(want[1][k], got[1][k]) for k in want[1])
    torch.cuda.synchronize()
    t = {k: v.requires_grad_(True) for k, v in t.items()}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = S.gated_linear(**t)
        grads = torch.autograd.grad(out, list(t.values()), d_out)
    for replay in range(4):
        say("replay", replay)
        new, new_d = make((rows, 96), 136, BF16, seed=20 + replay)
        with torch.no_grad():
            for k, v in t.items():
                v.copy_(new[k])
            d_out.copy_(new_d)
        graph.replay()
        torch.cuda.synchronize()
        want = run(new, new_d)
        assert torch.equal(out, want[0]) and all(torch.equal(g, want[1][k]) for g, k in zip(grads, NAMES))


def test_captured_with_gradients_beside_an_eager_graph_is_refused():
    t, d_out = make((7, 96), 136, BF16, seed=26)
    x = t["x"].requires_grad_(True)
    eager = S.gated_linear(x, t["w_gate"], t["w_up"])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        d_out * 2.0
        with pytest.raises(RuntimeError, match="default stream"):
            S.gated_linear(x, t["w_gate"], t["w_up"])
    del eager


def test_refusals():
    x, w, b = torch.zeros(4, 8, device="cuda"), torch.zeros(6, 8, device="cuda"), torch.zeros(6, device="cuda")
    f = S.gated_linear
    for call in (lambda: f(x, w[:, :4].contiguous(), w), lambda: f(x, w, w[:3]), lambda: f(x, w, w, b_gate=b[:3]),
                 lambda: f(x, w, w, b_up=b.view(1, 6)), lambda: f(x.t(), w, w), lambda: f(x, w.t(), w),
                 lambda: f(x, w, w, act="relu"), lambda: f(x[:, :0], w[:, :0], w[:, :0]), lambda: f(x, w[:0], w[:0]),
                 lambda: f(x[0, 0], w, w)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: f(x, w.half(), w), lambda: f(x, w, w, b_gate=b.half()), lambda: f(x.cpu(), w, w),
                 lambda: f(x, w.cpu(), w), lambda: f(x.double(), w.double(), w.double())):
        with pytest.raises(TypeError):
            call()
    a = x.clone().requires_grad_(True)
    with pytest.raises(RuntimeError, match="create_graph"):
        torch.autograd.grad(f(a, w, w).sum(), a, create_graph=True)
