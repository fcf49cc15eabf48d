"""The joint between two blocks on the GPU, forward and gradients, against the
oracle in 64 bits (bounds: train_oracle)."""
import math

import pytest
import torch

import ssim_loss_amd as S
from gpu_util import say
from train_oracle import Joint, check, joint

pytestmark = pytest.mark.gpu
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
TYPES = [(F32, F32), (F16, F16), (BF16, BF16), (F32, F16), (F32, BF16)]  # x, branch
NAMES = ("x", "branch", "gate", "scale", "post_weight", "pre_weight")


def make(shape, types, gate=None, act="none", weights=True, seed=0, offset=0):
    """Inputs with gradients wanted; `offset` starts each tensor that many
    elements into its memory."""
    rng = torch.Generator(device="cuda").manual_seed(seed)

    def n(size, dtype, std=1.0, mean=0.0):
        count = math.prod(size)
        flat = (torch.randn(count + offset, generator=rng, device="cuda") * std + mean).to(dtype)
        return flat[offset:].view(size)

    d = shape[-1]
    t = {"x": n(shape, types[0], 2.0), "branch": n(shape, types[1], 0.7, 0.1),
         "gate": None if gate is None else n(gate, types[1]),
         "scale": n((d,), F32, 0.3, 0.5) if weights else None,
         "post_weight": n((d,), F32, 0.1, 1.0) if weights else None,
         "pre_weight": n((d,), F32, 0.1, 1.0) if weights else None}
    t = {k: v.detach().requires_grad_(True) if v is not None else None for k, v in t.items()}
    return t, n(shape, types[0], 0.1), n(shape, types[1], 0.1), act


def run(t, dr, dh, act, eps=1e-6, leaves=NAMES):
    leaves = [k for k in leaves if t[k] is not None]
    r, h = S.block_norm(t["x"], t["branch"], gate=t["gate"], scale=t["scale"],
                        post_weight=t["post_weight"], pre_weight=t["pre_weight"], eps=eps,
                        gate_act=act)
    outs, ups = zip(*[(o, u) for o, u in ((r, dr), (h, dh)) if u is not None])
    grads = torch.autograd.grad(outs, [t[k] for k in leaves], ups)
    return r.detach(), h.detach(), dict(zip(leaves, grads))


def verify(made, eps=1e-6):
    t, dr, dh, act = made
    r, h, grads = run(t, dr, dh, act, eps)
    torch.cuda.synchronize()
    want = Joint(*t.values(), eps, act, dr, dh)
    check(r, *want.residual, "residual")
    check(h, *want.normed, "normed")
    for k, g in grads.items():
        assert g.dtype == t[k].dtype
        check(g, *want.grads[k], f"gradient of {k}")
    # the call without gradients is the same forward
    with torch.no_grad():
        r2, h2 = S.block_norm(t["x"], t["branch"], t["gate"], t["scale"], t["post_weight"],
                              t["pre_weight"], eps, act)
    assert torch.equal(r, r2) and torch.equal(h, h2)
    return r, h, grads


# around a thread's vector, a wave's row in one and two vectors, a workgroup's
# row in one, two, four and eight, and the widest
WIDTHS = [1, 2, 7, 8, 9, 48, 255, 256, 257, 384, 511, 513, 640, 1001, 1024, 1025, 1153, 2048, 2049,
          4095, 4097, 8191, 8193, 16384]


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("width", WIDTHS)
def test_widths(width, types):
    say("joint", width, types)
    verify(make((5, width), types, gate=(5, width), act="sigmoid", seed=width))


@pytest.mark.parametrize("types", [(F32, F32), (BF16, BF16), (F32, F16)])
@pytest.mark.parametrize("width", [9, 640, 1153, 4097, 8193])
@pytest.mark.parametrize("gate", ["none", "sample", "whole"])
def test_shared_gates_and_none(gate, width, types):
    shape = (3, 11, width)
    g = {"none": None, "sample": (3, 1, width), "whole": (1, 1, width)}[gate]
    say("joint", gate, width, types)
    verify(make(shape, types, gate=g, act="sigmoid", seed=width + 1))
    verify(make(shape, types, gate=g, act="none", seed=width + 2))


@pytest.mark.parametrize("shape,gate", [
    ((1, 1, 64), (1, 1, 64)),          # one token
    ((64,), None),
    ((6000, 2, 64), (6000, 1, 64)),    # more gate rows than workgroups: groups are not cut
    ((1500, 3, 1100), (1500, 1, 1100)),
    ((2, 3001, 72), (2, 1, 72)),       # few: cut into many parts
    ((2, 901, 1200), (2, 1, 1200)),
    ((7, 5, 3, 100), (7, 5, 1, 100)),
    ((7, 5, 3, 100), (7, 1, 1, 100)),
    ((5000, 72), (5000, 72)),          # more rows than workgroups
    ((3000, 1200), None),
    ((300, 2, 8200), (300, 1, 8200)),  # rows loaded twice: several groups to a workgroup
    ((2, 300, 8200), (2, 1, 8200)),
    ((600, 8200), (600, 8200)),
])
@pytest.mark.parametrize("types", [(F32, F32), (F32, BF16)])
def test_rows_and_groups(shape, gate, types):
    say("joint", shape, gate, types)
    verify(make(shape, types, gate=gate, act="sigmoid", seed=40))


# rows that 8, 16, 32 and 64 lanes take, in either type, with several to a wave:
# rows left over in the last one, groups that end inside one
@pytest.mark.parametrize("types", [(F32, F32), (BF16, BF16), (F32, F16)])
@pytest.mark.parametrize("width", [3, 31, 32, 33, 63, 64, 65, 127, 128, 129, 256, 257])
def test_several_rows_to_a_wave(width, types):
    say("joint", width, types)
    verify(make((2, 1301, width), types, gate=(2, 1301, width), act="sigmoid", seed=width))
    verify(make((3, 75, width), types, gate=(3, 1, width), act="sigmoid", seed=width + 1))
    verify(make((1500, 3, width), types, gate=(1500, 1, width), seed=width + 2))


@pytest.mark.parametrize("types", [(F32, F32), (F16, F16), (F32, BF16)])
@pytest.mark.parametrize("width", [640, 1153, 2048])
def test_tensors_that_start_anywhere(width, types):
    verify(make((4, width), types, gate=(4, width), seed=41, offset=1))
    verify(make((2, 3, width), types, gate=(2, 1, width), seed=42, offset=3))


@pytest.mark.parametrize("width", [100, 2000])
def test_without_weights(width):
    verify(make((9, width), (BF16, BF16), weights=False, seed=43))
    verify(make((9, width), (F32, F32), gate=(9, width), weights=False, seed=44))


@pytest.mark.parametrize("gate", [None, (2, 6, 300), (2, 1, 300)])
def test_any_set_of_leaves(gate):
    """Gradients that are not wanted are not formed; the others keep their bits."""
    t, dr, dh, act = make((2, 6, 300), (F32, BF16), gate=gate, act="sigmoid", seed=45)
    all_of = run(t, dr, dh, act)[2]
    for leaf in all_of:
        for k, v in t.items():
            if v is not None:
                v.requires_grad_(k == leaf)
        assert torch.equal(run(t, dr, dh, act, leaves=[leaf])[2][leaf], all_of[leaf]), leaf


@pytest.mark.parametrize("width", [300, 1300])
@pytest.mark.parametrize("which", ["residual", "normed"])
def test_one_upstream_gradient_alone(which, width):
    t, dr, dh, act = make((7, width), (BF16, BF16), gate=(7, width), seed=46)
    verify((t, dr if which == "residual" else None, dh if which == "normed" else None, act))


def test_upstream_gradients_that_are_not_contiguous():
    t, _, _, act = make((4, 6, 200), (F32, F32), seed=47)
    r, h = S.block_norm(t["x"], t["branch"], pre_weight=t["pre_weight"])
    (r.sum() + (h.transpose(0, 1) * 2.0).sum()).backward()
    one = torch.ones_like(r)
    want = Joint(t["x"], t["branch"], None, None, None, t["pre_weight"], 1e-6, act, one, 2 * one)
    check(t["x"].grad, *want.grads["x"], "x")
    check(t["pre_weight"].grad, *want.grads["pre_weight"], "pre_weight")


@pytest.mark.parametrize("types", [(F32, F32), (F16, F16)])
def test_rows_of_zeros(types):
    """A row that a mask has emptied: its root is that of eps."""
    made = make((6, 500), types, gate=(6, 500), seed=48)
    with torch.no_grad():
        made[0]["branch"][1] = 0
        made[0]["x"][2] = 0
        made[0]["branch"][2] = 0
    r, h, grads = verify(made, eps=1e-2)
    assert not r[2].any() and not h[2].any()
    assert all(torch.isfinite(g).all() for g in grads.values())


@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("width", [500, 3000])
def test_a_row_that_is_not_finite_stays_alone(bad, width):
    made = make((9, width), (BF16, BF16), gate=(9, width), seed=49)
    clean = run(*made)
    with torch.no_grad():
        made[0]["branch"][4, 17] = bad
    r, h, grads = run(*made)
    others = [k for k in range(9) if k != 4]
    for a, b in ((r, clean[0]), (h, clean[1]), (grads["x"], clean[2]["x"]),
                 (grads["branch"], clean[2]["branch"]), (grads["gate"], clean[2]["gate"])):
        assert torch.equal(a[others], b[others])
    assert torch.isnan(h[4]).any()
    assert torch.isnan(grads["scale"]).any()


@pytest.mark.parametrize("types", [(F32, F32), (F16, F16), (F32, BF16)])
def test_gates_at_the_ends_of_the_sigmoid(types):
    made = make((3, 700), types, gate=(3, 700), act="sigmoid", seed=50)
    with torch.no_grad():
        made[0]["gate"][0] = 200.0
        made[0]["gate"][1] = -200.0
        made[0]["gate"][2, ::2] = math.inf
        made[0]["gate"][2, 1::2] = -math.inf
    r, h, grads = run(*made)
    x, b = made[0]["x"].detach(), made[0]["branch"].detach()
    assert torch.equal(r[1], x[1]) and torch.equal(r[2, 1::2], x[2, 1::2])
    assert not torch.equal(r[0], x[0])
    assert not grads["gate"][1:].any() and all(torch.isfinite(g).all() for g in grads.values())


@pytest.mark.parametrize("rows", [(0, 8), (2, 0, 8)])
def test_no_rows(rows):
    t, dr, dh, act = make(rows, (F32, BF16), gate=(2, 1, 8) if len(rows) == 3 else None, seed=51)
    r, h, grads = run(t, dr, dh, act)
    assert r.shape == h.shape == rows and r.dtype == F32 and h.dtype == BF16
    for k, g in grads.items():
        assert g.shape == t[k].shape and not g.any()


def test_the_same_bits_again():
    made = make((2, 700, 1001), (F16, F16), gate=(2, 1, 1001), act="sigmoid", seed=52)
    a, b = run(*made), run(*made)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert all(torch.equal(a[2][k], b[2][k]) for k in a[2])


def test_gradients_are_the_definitions_differences():
    """The kernels' gradients along a direction against differences of the
    definition in 64 bits, within the gradients' own bounds."""
    t, dr, dh, act = make((3, 4, 37), (F32, F32), gate=(3, 1, 37), act="sigmoid", seed=53)
    grads = run(t, dr, dh, act)[2]
    want = Joint(*t.values(), 1e-6, act, dr, dh)
    wide = {k: v.detach().cpu().double() for k, v in t.items()}
    ups = [u.cpu().double() for u in (dr, dh)]
    f = lambda v: sum((o * u).sum() for o, u in zip(joint(*v.values(), 1e-6, act), ups))
    rng = torch.Generator().manual_seed(54)
    step = 1e-5
    for k, v in wide.items():
        along = torch.randn(v.shape, generator=rng, dtype=torch.float64)
        up, down = ({**wide, k: v + s * along} for s in (step, -step))
        slope = (f(up) - f(down)) / (2 * step)
        got = (grads[k].cpu().double() * along).sum()
        bound = (want.grads[k][1] * along.abs()).sum() + 1e-7 * (1 + abs(slope))
        assert abs(got - slope) <= bound, k


def test_past_32_bit_offsets():
    rows, width = (1 << 31) // 2048 + 3, 2048
    x = torch.zeros(rows, width, dtype=BF16, device="cuda")
    branch = torch.zeros_like(x)
    rng = torch.Generator(device="cuda").manual_seed(55)
    some = [0, (1 << 30) // width, (1 << 31) // width - 1, (1 << 31) // width, rows - 1]
    for k in some:
        x[k] = torch.randn(width, generator=rng, device="cuda").bfloat16()
        branch[k] = torch.randn(width, generator=rng, device="cuda").bfloat16()
    say("joint", rows, width)
    x.requires_grad_(True)
    branch.requires_grad_(True)
    r, h = S.block_norm(x, branch)
    gx, gb = torch.autograd.grad((r, h), (x, branch), (x.detach(), branch.detach()))
    pick = lambda t: t.detach()[torch.tensor(some, device="cuda")]
    want = Joint(pick(x), pick(branch), None, None, None, None, 1e-6, "none", pick(x), pick(branch))
    check(pick(r), *want.residual, "residual")
    check(pick(h), *want.normed, "normed")
    check(pick(gx), *want.grads["x"], "gradient of x")
    check(pick(gb), *want.grads["branch"], "gradient of branch")
    assert int(r.count_nonzero(1).ne(0).sum()) == len(some)


def test_on_another_stream():
    made = make((900, 1024), (BF16, BF16), gate=(900, 1024), seed=56)
    want = run(*made)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = run(*made)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    assert all(torch.equal(want[2][k], got[2][k]) for k in want[2])


@pytest.mark.parametrize("gate", [(2, 150, 520), (2, 1, 520)])
def test_captured_in_a_graph(gate):
    """Forward and gradients in one graph, replayed on new inputs, against the
    eager call after each replay."""
    t, dr, dh, act = make((2, 150, 520), (F32, BF16), gate=gate, act="sigmoid", seed=57)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run(t, dr, dh, act)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r, h, grads = run(t, dr, dh, act)
    for replay in range(4):
        say("replay", replay)
        new = make((2, 150, 520), (F32, BF16), gate=gate, act="sigmoid", seed=60 + replay)
        with torch.no_grad():
            for k, v in t.items():
                v.copy_(new[0][k])
            dr.copy_(new[1])
            dh.copy_(new[2])
        graph.replay()
        torch.cuda.synchronize()
        r2, h2, grads2 = run(*new)
        assert torch.equal(r, r2) and torch.equal(h, h2)
        assert all(torch.equal(grads[k], grads2[k]) for k in grads)


def test_captured_with_gradients_beside_an_eager_graph_is_refused():
    """The leaves' nodes belong to the default stream as long as the eager
    graph lives; afterwards the same capture is taken."""
    t, dr, dh, act = make((3, 40), (F32, F32), gate=(3, 40), seed=70)
    want = run(t, dr, dh, act)
    call = lambda: S.block_norm(t["x"], t["branch"], t["gate"], t["scale"], t["post_weight"],
                                t["pre_weight"], 1e-6, act)
    eager = call()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dr * 2.0
        with pytest.raises(RuntimeError, match="default stream"):
            call()
        with torch.no_grad():
            r, h = call()
    say("captured")
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(r, want[0]) and torch.equal(h, want[1])
    del eager
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run(t, dr, dh, act)
    for replay in range(3):
        say("replay", replay)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        assert all(torch.equal(got[2][k], want[2][k]) for k in want[2])


def test_two_passes_through_one_graph():
    t, dr, dh, act = make((3, 40), (F32, F32), seed=71)
    r, h = S.block_norm(t["x"], t["branch"], scale=t["scale"])
    leaves = [t["x"], t["branch"], t["scale"]]
    a = torch.autograd.grad((r, h), leaves, (dr, dh), retain_graph=True)
    b = torch.autograd.grad((r, h), leaves, (dr, dh))
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    with pytest.raises(RuntimeError, match="second time"):
        torch.autograd.grad((r, h), leaves, (dr, dh))


def test_refusals():
    x = torch.ones(2, 3, 8, device="cuda")
    w = torch.ones(8, device="cuda")
    f = S.block_norm
    for call in (lambda: f(x, x[:1]), lambda: f(x.transpose(0, 1), x.transpose(0, 1)),
                 lambda: f(x, x, gate=w), lambda: f(x, x, gate=torch.ones(1, 3, 8, device="cuda")),
                 lambda: f(x, x, gate=torch.ones(2, 3, 4, device="cuda")),
                 lambda: f(x, x, scale=w[:4]), lambda: f(x, x, pre_weight=w.view(1, 8)),
                 lambda: f(x, x, eps=-1.0), lambda: f(x, x, eps=math.nan),
                 lambda: f(x, x, gate_act="relu"), lambda: f(w[0], w[0]),
                 lambda: f(torch.ones(2, 16385, device="cuda"), torch.ones(2, 16385, device="cuda"))):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: f(x, x.cpu()), lambda: f(x.half(), x), lambda: f(x.half(), x.bfloat16()),
                 lambda: f(x.double(), x.double()), lambda: f(x, x, gate=x.half()),
                 lambda: f(x, x, scale=w.half()), lambda: f(x, x, scale=w.cpu())):
        with pytest.raises(TypeError):
            call()
    with pytest.raises(S.TrainError) as e:  # a number, but none of fp32
        f(x, x, eps=1e300)
    assert e.value.code == -10
    a = x.clone().requires_grad_(True)
    r, h = f(a, x)
    with pytest.raises(RuntimeError, match="create_graph"):
        torch.autograd.grad(h.sum(), a, create_graph=True)
    saved = f(a, x.requires_grad_(True))[1].sum()
    with torch.no_grad():
        a += 1
    with pytest.raises(RuntimeError, match="modified"):
        saved.backward()
