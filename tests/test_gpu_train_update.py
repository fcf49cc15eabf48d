"""Clipping by the global norm and AdamW on the GPU against the oracle in 64
bits (bounds: train_oracle)."""
import math

import pytest
import torch

import ssim_loss_amd as S
from gpu_util import say
from train_oracle import U, adamw, check, check_norm, clipped, factor, norm_of

pytestmark = pytest.mark.gpu
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


def _values(rng, n, dtype, std=1.0):
    return (torch.randn(n, generator=rng, device="cuda") * std).to(dtype)


def _list(sizes, dtypes, seed, std=1.0):
    rng = torch.Generator(device="cuda").manual_seed(seed)
    return [_values(rng, n, dtypes[k % len(dtypes)], std) for k, n in enumerate(sizes)]


def _packed(sizes, dtype, seed, offset=0, std=1.0):
    rng = torch.Generator(device="cuda").manual_seed(seed)
    flat = _values(rng, offset + sum(sizes) + 5, dtype, std)
    out, at = [], offset
    for n in sizes:
        out.append(flat[at:at + n])
        at += n
    return flat, out


def _check_clip(grads, max_norm, out=None):
    before = [g.clone() for g in grads]
    got = S.clip_grads_(grads, max_norm, out=out)
    torch.cuda.synchronize()
    cpu = [b.cpu() for b in before]
    norm = norm_of(cpu)
    check_norm(got, norm)
    c = factor(norm, max_norm)
    for k, (g, b) in enumerate(zip(out or grads, cpu)):
        check(g, *clipped(b, c), f"tensor {k}")
    if out is not None:
        assert all(torch.equal(g, b) for g, b in zip(grads, before))
    return got


# one element; around a thread's vector, a workgroup's chunk and its multiples; several chunks
SIZES = [1, 3, 4, 5, 7, 8, 9, 255, 1023, 1024, 1025, 2047, 2048, 2049, 4095, 4097, 8193, 100003]


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("n", SIZES)
def test_clip_one_tensor(n, dtype, in_place):
    say("clip", n, dtype, in_place)
    grads = _list([n], [dtype], n)
    out = None if in_place else [torch.full_like(g, float("nan")) for g in grads]
    _check_clip(grads, 0.5, out)


def test_clip_a_mixed_list_and_the_norm_alone():
    grads = _list([5, 0, 4097, 1, 20000, 333], [F32, BF16, F16], 5)
    alone = S.grad_norm(grads)
    got = _check_clip(grads, 2.0)
    assert torch.equal(alone, got)


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("offset", [0, 1, 3])
def test_clip_packed_tensors_leave_their_neighbours_alone(dtype, offset):
    """Tensors packed end to end at odd places (one run of memory), in place
    and into tensors that start at another alignment."""
    sizes = [7, 1, 1000, 4096, 13]
    flat, grads = _packed(sizes, dtype, 6, offset)
    before = flat.clone()
    to, out = _packed(sizes, dtype, 7, (offset + 2) % 4)
    edge = to.clone()
    _check_clip(grads, 1.0, out)
    first = (offset + 2) % 4
    assert torch.equal(to[:first], edge[:first])
    assert torch.equal(to[first + sum(sizes):], edge[first + sum(sizes):])
    _check_clip(grads, 1.0)
    assert torch.equal(flat[:offset], before[:offset])
    assert torch.equal(flat[offset + sum(sizes):], before[offset + sum(sizes):])


def test_clip_more_tensors_than_a_launch_holds():
    sizes = [1 + 37 * k % 501 for k in range(700)]
    _check_clip(_list(sizes, [F32, BF16, F16], 8), 1.0)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("sizes", [[1, 2, 3, 1, 3, 45], [4096] * 8, [32768], [32769], [4097] * 8,
                                   [1] * 8, [1] * 9, [5, 32000, 7], [16384, 16384]])
def test_clip_few_gradients(sizes, dtype):
    """Lists at and around what one launch takes, out of place in one
    workgroup and in several, and in place."""
    say("clip", sizes, dtype)
    grads = _list(sizes, [dtype], 15)
    _check_clip(grads, 0.5, [torch.full_like(g, float("nan")) for g in grads])
    _check_clip(grads, 0.25)


def test_clip_large_lists_take_the_large_chunks():
    """More than the last-level cache holds twice over, in both types."""
    _check_clip(_list([50_000_001, 90_000_003], [F32, BF16], 9), 1.0)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_clip_below_the_threshold_changes_nothing(dtype):
    grads = _list([5000], [dtype], 10, std=1e-4)
    before = grads[0].clone()
    S.clip_grads_(grads, 1.0)
    assert torch.equal(grads[0], before)
    out = [torch.zeros_like(before)]
    S.clip_grads_(grads, 1.0, out=out)
    assert torch.equal(out[0], before)


def test_clip_to_zero():
    grads = _list([1000], [F32], 11)
    S.clip_grads_(grads, 0.0)
    assert not grads[0].any()


@pytest.mark.parametrize("size", [1e-30, 1e25])
def test_norm_of_gradients_whose_squares_leave_fp32(size):
    grads = _list([3000], [F32], 12, std=size)
    check_norm(S.grad_norm(grads), norm_of([g.cpu() for g in grads]))
    _check_clip(_list([3000], [BF16], 12, std=size), 1.0)


@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_clip_of_gradients_that_are_not_finite_follows_the_formula(bad):
    grads = _list([2000, 300], [F32, F16], 13)
    grads[0][77] = bad
    want = norm_of([g.cpu() for g in grads])
    c = factor(want, 1.0).float()
    expect = [(g.float().cpu() * c).to(g.dtype) for g in grads]
    got = S.clip_grads_(grads, 1.0)
    assert torch.equal(got.cpu(), want.float()) or (math.isnan(want) and math.isnan(got))
    for g, e in zip(grads, expect):
        assert torch.equal(torch.isnan(g.cpu()), torch.isnan(e))
        assert torch.equal(torch.nan_to_num(g.cpu()), torch.nan_to_num(e))


def test_clip_gives_the_same_bits_again_and_for_any_grouping_of_outputs():
    grads = _list([70001, 4099], [BF16, F32], 14)
    outs = [[torch.empty_like(g) for g in grads] for _ in range(2)]
    norms = [S.clip_grads_(grads, 0.1, out=o) for o in outs]
    assert torch.equal(*norms)
    for a, b in zip(*outs):
        assert torch.equal(a, b)


def test_clip_past_32_bit_offsets():
    n = (1 << 32) + 9
    g = torch.zeros(n, dtype=BF16, device="cuda")
    places = [0, 12345, (1 << 31) - 1, 1 << 31, (1 << 32) - 3, 1 << 32, n - 1]
    for k, at in enumerate(places):
        g[at] = k + 1.0
    say("clip", n)
    got = S.clip_grads_([g], 1.0)
    norm = math.sqrt(sum((k + 1.0) ** 2 for k in range(len(places))))
    check_norm(got, torch.tensor(norm, dtype=torch.float64))
    want = torch.tensor([k + 1.0 for k in range(len(places))]).bfloat16()
    bits, bound = clipped(want, torch.tensor(1.0 / (norm + 1e-6), dtype=torch.float64))
    check(g[torch.tensor(places, device="cuda")], bits, bound, "far elements")
    assert int(torch.count_nonzero(g)) == len(places)


def test_clip_refusals():
    a = torch.ones(8, 8, device="cuda")
    for call in (lambda: S.clip_grads_([a[:, :4]], 1.0),
                 lambda: S.clip_grads_([a], 1.0, out=[a[:4]]),
                 lambda: S.clip_grads_([a], 1.0, out=[torch.ones(8, 8, device="cuda").t()]),
                 lambda: S.clip_grads_([a], -1.0)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: S.clip_grads_([a.double()], 1.0), lambda: S.clip_grads_([a, a.cpu()], 1.0),
                 lambda: S.clip_grads_([a], 1.0, out=[a.half()])):
        with pytest.raises(TypeError):
            call()
    for call in (lambda: S.clip_grads_([a, a], 1.0), lambda: S.clip_grads_([a, a[2:4]], 1.0),
                 lambda: S.clip_grads_([a[:7]], 1.0, out=[a[1:]])):
        with pytest.raises(S.TrainError) as e:
            call()
        assert e.value.code == -5
    assert torch.equal(a, torch.ones_like(a))


# ------------------------------------------------------------------ AdamW
LR, B1, B2, EPS, DECAY = 2e-3, 0.9, 0.97, 1e-8, 0.02


class Net:
    """Parameters with state and gradients, and their copies on the CPU."""

    def __init__(self, sizes, dtype, masters, seed, grad_dtype=None, packed=None):
        rng = torch.Generator(device="cuda").manual_seed(seed)
        total = sum(sizes)

        def cut(flat):
            out, at = [], packed or 0
            for n in sizes:
                out.append(flat[at:at + n])
                at += n
            return out if packed is not None else [t.clone() for t in out]

        room = total + (packed or 0)
        w = _values(rng, room, F32, 0.05)
        self.params = cut(w.to(dtype) if dtype != F32 else w.clone())
        self.masters = cut(w) if masters else None
        self.m = cut(_values(rng, room, F32, 1e-3))
        self.v = cut(torch.rand(room, generator=rng, device="cuda") * 1e-5)
        self.grads = cut(_values(rng, room, grad_dtype or dtype, 0.03))

    def cpu(self):
        f = lambda ts: None if ts is None else [t.cpu().clone() for t in ts]
        return f(self.params), f(self.masters), f(self.m), f(self.v), f(self.grads)

    def optimizer(self, max_norm=1.0, step=3, lr=LR):
        return S.AdamW(self.params, lr=lr, betas=(B1, B2), eps=EPS, weight_decay=DECAY,
                       max_norm=max_norm, exp_avgs=self.m, exp_avg_sqs=self.v,
                       masters=self.masters, step=step)


def _check_update(net, before, norm, max_norm, t, lr=LR):
    params, masters, m, v, grads = before
    c = torch.ones((), dtype=torch.float64)
    if max_norm is None:
        assert norm is None
    else:
        want = norm_of(grads)
        check_norm(norm, want)
        c = factor(want, max_norm)
    for k in range(len(params)):
        p, w, m1, v1 = adamw(params[k], masters[k] if masters else None, m[k], v[k], grads[k], c,
                             lr, B1, B2, EPS, DECAY, t)
        check(net.params[k], *p, f"parameter {k}")
        if masters:
            check(net.masters[k], *w, f"master {k}")
        check(net.m[k], *m1, f"exp_avg {k}")
        check(net.v[k], *v1, f"exp_avg_sq {k}")
    for g, b in zip(net.grads, grads):
        assert torch.equal(g.cpu(), b)


@pytest.mark.parametrize("max_norm", [1.0, 0.01, None])
@pytest.mark.parametrize("dtype,masters,grad", [(F32, False, None), (F32, True, None),
                                                (BF16, True, None), (F16, True, None),
                                                (BF16, False, None), (F16, False, None),
                                                (BF16, True, F32), (F16, False, F32)])
def test_adamw_types(dtype, masters, grad, max_norm):
    say("adamw", dtype, masters, grad, max_norm)
    net = Net([1, 1000, 37, 4099], dtype, masters, 20, grad)
    before = net.cpu()
    opt = net.optimizer(max_norm)
    norm = opt.step(net.grads)
    assert opt.steps == 4
    _check_update(net, before, norm, max_norm, 4)


@pytest.mark.parametrize("sizes", [[1], [2, 3], [1023, 1025], [2049], [0, 5], [9000]])
@pytest.mark.parametrize("packed", [None, 0, 1, 3])
def test_adamw_sizes_and_places(sizes, packed):
    net = Net(sizes, BF16, True, 21, packed=packed)
    before = net.cpu()
    _check_update(net, before, net.optimizer().step(net.grads), 1.0, 4)


def test_adamw_more_tensors_than_a_launch_holds():
    net = Net([1 + 53 * k % 301 for k in range(200)], F32, False, 22)
    before = net.cpu()
    _check_update(net, before, net.optimizer().step(net.grads), 1.0, 4)


@pytest.mark.parametrize("dtype,masters,grad", [(F32, False, None), (BF16, True, None),
                                                (F16, False, F32), (F16, True, F32)])
@pytest.mark.parametrize("sizes", [[1, 2, 3, 1, 3, 45], [32768], [32769], [4093] * 8, [1] * 9])
@pytest.mark.parametrize("max_norm", [0.5, None])
def test_adamw_few_parameters(sizes, dtype, masters, grad, max_norm):
    """Lists at and around what one launch takes; two updates, so that the
    count that the workgroups keep is used twice."""
    say("adamw", sizes, dtype, masters, grad)
    net = Net(sizes, dtype, masters, 32, grad)
    opt = net.optimizer(max_norm)
    for t in (4, 5):
        before = net.cpu()
        _check_update(net, before, opt.step(net.grads), max_norm, t)
    assert opt._step.tolist() == [5, 0]


def test_adamw_large_lists_take_the_large_chunks():
    net = Net([20_000_003, 500_001], F16, True, 23)
    before = net.cpu()
    _check_update(net, before, net.optimizer().step(net.grads), 1.0, 4)


def test_adamw_from_nothing_over_several_steps():
    """Zero states and no updates before: the bias corrections are largest."""
    rng = torch.Generator(device="cuda").manual_seed(24)
    p = [_values(rng, 3001, F32)]
    opt = S.AdamW(p, lr=LR, betas=(B1, B2), eps=EPS, weight_decay=DECAY)
    for t in range(1, 4):
        net = Net.__new__(Net)
        net.params, net.masters, net.m, net.v = p, None, opt.exp_avgs, opt.exp_avg_sqs
        net.grads = [_values(rng, 3001, F32, 0.1)]
        before = net.cpu()
        _check_update(net, before, opt.step(net.grads), None, t)
    assert opt.steps == 3


def test_adamw_takes_the_parameters_gradients_and_skips_missing_ones():
    net = Net([500, 600], F32, False, 25)
    net.params[0].grad = net.grads[0]
    before = net.cpu()
    opt = net.optimizer(max_norm=0.1)
    norm = opt.step()
    check_norm(norm, norm_of(before[4][:1]))
    kept = [net.params[1], net.m[1], net.v[1]]
    for now, was in zip(kept, (before[0][1], before[2][1], before[3][1])):
        assert torch.equal(now.cpu(), was)
    assert not torch.equal(net.params[0].cpu(), before[0][0])
    opt.zero_grad()
    assert float(opt.step()) == 0.0 and opt.steps == 5


def test_adamw_learning_rate_on_the_device_and_changed_on_the_host():
    net, other = Net([5000], F32, False, 26), Net([5000], F32, False, 26)
    lr = torch.tensor(0.25, device="cuda")  # exact in fp32
    a, b = net.optimizer(lr=lr), other.optimizer(lr=0.25)
    a.step(net.grads)
    b.step(other.grads)
    assert torch.equal(net.params[0], other.params[0])
    lr.fill_(0.125)
    b.lr = 0.125
    a.step(net.grads)
    b.step(other.grads)
    assert torch.equal(net.params[0], other.params[0])


def test_adamw_state_dict_goes_on_where_it_was():
    net = Net([700, 20], BF16, True, 27)
    opt = net.optimizer()
    opt.step(net.grads)
    state, params = opt.state_dict(), [p.clone() for p in net.params]
    opt.step(net.grads)
    again = S.AdamW(params, lr=LR, betas=(B1, B2), eps=EPS, weight_decay=DECAY, max_norm=1.0,
                    masters=[p.float() for p in params])
    again.load_state_dict(state)
    assert again.steps == 4
    again.step(net.grads)
    for a, b in zip(net.params + net.masters + net.m, params + again.masters + again.exp_avgs):
        assert torch.equal(a, b)
    with pytest.raises(ValueError):
        again.load_state_dict({**state, "masters": None})


def test_adamw_marks_its_tensors_as_written():
    net = Net([100], F32, False, 28)
    versions = [t._version for t in (net.params[0], net.m[0], net.v[0])]
    net.optimizer().step(net.grads)
    assert all(t._version > v for t, v in zip((net.params[0], net.m[0], net.v[0]), versions))


def test_adamw_refusals():
    p = torch.zeros(8, device="cuda")
    g = torch.ones(8, device="cuda")
    a = torch.zeros(4, 2, device="cuda").t()
    for make in (lambda: S.AdamW([p], lr=-1.0), lambda: S.AdamW([p], betas=(1.0, 0.9)),
                 lambda: S.AdamW([p], eps=-1.0), lambda: S.AdamW([p], max_norm=math.nan),
                 lambda: S.AdamW([p], exp_avgs=[]), lambda: S.AdamW([p], step=-1),
                 lambda: S.AdamW([a]).step([torch.ones(2, 4, device="cuda")]),
                 lambda: S.AdamW([a], exp_avgs=[torch.zeros(8, device="cuda")]).step([a.clone()]),
                 lambda: S.AdamW([p]).step([g, g]), lambda: S.AdamW([p]).step([g[:4]]),
                 lambda: S.AdamW([torch.zeros(4, 4, device="cuda").t()]).step([g.view(2, 4)])):
        with pytest.raises(ValueError):
            make()
    for make in (lambda: S.AdamW([p]).step([g.half()]), lambda: S.AdamW([p]).step([g.cpu()]),
                 lambda: S.AdamW([p], masters=[p.half()]).step([g]),
                 lambda: S.AdamW([p], exp_avgs=[p.double()]).step([g]),
                 lambda: S.AdamW([p], lr=torch.tensor(0.1)).step([g])):
        with pytest.raises(TypeError):
            make()
    for make in (lambda: S.AdamW([p, p]).step([g, g.clone()]),
                 lambda: S.AdamW([p], masters=[p]).step([g]), lambda: S.AdamW([p]).step([p])):
        with pytest.raises(S.TrainError) as e:
            make()
        assert e.value.code == -5
    assert not p.any()


def test_update_on_another_stream_runs_there():
    net, other = Net([300_000], BF16, True, 29), Net([300_000], BF16, True, 29)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(5):
            net.optimizer().step(net.grads)
    torch.cuda.current_stream().wait_stream(side)
    for _ in range(5):
        other.optimizer().step(other.grads)
    for a, b in zip(net.params + net.masters, other.params + other.masters):
        assert torch.equal(a, b)


def test_update_captured_in_a_graph_follows_its_step_and_rate():
    """Each replay is one more update, with the rate's present value; eager
    work and waits lie between the replays."""
    net, other = Net([30_000, 77], BF16, True, 30), Net([30_000, 77], BF16, True, 30)
    lr = torch.tensor(0.5, device="cuda")
    a, b = net.optimizer(lr=lr), other.optimizer(lr=lr)
    grads = [g.clone() for g in net.grads]
    scaled = [torch.empty_like(g) for g in grads]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):  # first use outside the capture
        S.clip_grads_(grads, 0.5, out=scaled)
        S.AdamW([torch.zeros(4, device="cuda")]).step([torch.zeros(4, device="cuda")])
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norm = S.clip_grads_(grads, 0.5, out=scaled)
        a.step(scaled)
    rng = torch.Generator(device="cuda").manual_seed(31)
    for replay in range(5):
        say("replay", replay)
        lr.fill_(0.5 / (replay + 1))
        for g in grads:
            g.copy_(_values(rng, g.numel(), g.dtype, 0.02))
        graph.replay()
        torch.cuda.synchronize()
        out = [torch.empty_like(g) for g in grads]
        want = S.clip_grads_(grads, 0.5, out=out)
        b.step(out)
        assert torch.equal(norm, want)
        assert a.steps == b.steps == 4 + replay
        for x, y in zip(net.params + net.masters + net.m + net.v,
                        other.params + other.masters + other.m + other.v):
            assert torch.equal(x, y)


@pytest.mark.parametrize("dtype,masters", [(F32, False), (BF16, True)])
def test_tensors_in_another_order_of_their_dimensions(dtype, masters):
    """Convolution weights in channels_last, beside a contiguous one: as their
    contiguous copies."""
    shapes = [(16, 8, 3, 3), (5, 1, 3, 3), (24, 7)]
    rng = torch.Generator(device="cuda").manual_seed(33)
    last = lambda t: t.to(memory_format=torch.channels_last) if t.dim() == 4 else t.t().contiguous().t()
    made = [_values(rng, math.prod(s), F32, 0.05).view(s) for s in shapes]
    grads = [_values(rng, math.prod(s), dtype).view(s) for s in shapes]
    sides = []
    for order in (last, lambda t: t.clone()):
        g = [order(t) for t in grads]
        params = [order(w.to(dtype)) for w in made]
        opt = S.AdamW(params, lr=LR, max_norm=0.5, masters=[order(w) for w in made] if masters else None)
        norm = [opt.step(g), opt.step(g)]
        clipped_to = [torch.zeros_like(t) for t in g]
        S.clip_grads_(g, 0.25, out=clipped_to)
        S.clip_grads_(g, 0.25)
        sides.append(norm + params + opt.exp_avgs + opt.exp_avg_sqs + (opt.masters or []) + clipped_to + g)
    assert not sides[0][2].is_contiguous() and sides[0][2].stride() == sides[0][5].stride()
    for a, b in zip(*sides):
        if a.dim():
            assert torch.equal(a, b)
        else:  # (squares are added in the order of the memory)
            check_norm(a, b.cpu().double())
