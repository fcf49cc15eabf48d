"""Clipping and AdamW, and what surrounds their launches."""
import pytest
import torch

import ssim_loss_amd as S
from gpu_util import say
from test_gpu_train_update import BF16, F16, F32, Net, _list, _values

pytestmark = pytest.mark.gpu


def test_an_error_left_by_another_call_is_not_this_ones():
    """The runtime keeps a refused call's error until somebody asks for it."""
    grads = _list([5000], [F32], 110)
    want = S.grad_norm(grads)
    torch.cuda.synchronize()
    hip = S.train.lib()  # (the runtime's functions are found through it)
    assert hip.hipSetDevice(1 << 20) != 0
    try:
        got = S.grad_norm(grads)
    finally:
        hip.hipGetLastError()
    assert torch.equal(got, want)


# past the single launch: by elements, by types, by runs, and past the tables of
# one launch (144 runs for the norm, 112 for clipping, 64 for AdamW)
LISTS = {"long": [300_000, 77], "nine": [501 + k for k in range(9)], "many": [1 + 37 * k % 501 for k in range(200)]}


class Several:
    """Nets of different types as one list."""

    def __init__(self, kinds, sizes):
        nets = [Net(sizes, *kind, 111 + k) for k, kind in enumerate(kinds)]
        self.params, self.m, self.v, self.grads = ([t for n in nets for t in getattr(n, name)]
                                                   for name in ("params", "m", "v", "grads"))
        self.masters = [t for n in nets for t in (n.masters or [None] * len(sizes))]

    def optimizer(self, lr, max_norm):
        return S.AdamW(self.params, lr=lr, betas=(0.9, 0.97), weight_decay=0.02, max_norm=max_norm,
                       exp_avgs=self.m, exp_avg_sqs=self.v, masters=self.masters, step=3)

    def state(self):
        return self.params + self.m + self.v + [w for w in self.masters if w is not None]


KINDS = {"fp32": [(F32, False)], "bf16": [(BF16, True)], "mixed": [(BF16, True), (F32, False), (F16, False)]}


@pytest.mark.parametrize("max_norm", [0.5, None])
@pytest.mark.parametrize("kinds", KINDS)
@pytest.mark.parametrize("sizes", LISTS)
def test_captured_updates_follow_their_step_and_rate(sizes, kinds, max_norm):
    """Clipping and an update in one graph, its rate on the device; eager work
    and waits lie between the replays, and each replay is the eager calls'."""
    say("captured", sizes, kinds, max_norm)
    made = lambda: Several(KINDS[kinds], LISTS[sizes])
    net, other = made(), made()
    lr = torch.tensor(0.5, device="cuda")
    a, b = net.optimizer(lr, max_norm), other.optimizer(lr, max_norm)
    grads = [g.clone() for g in net.grads]
    scaled = [torch.empty_like(g) for g in grads]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):  # first use outside the capture
        S.clip_grads_(grads, 0.5, out=scaled)
        made().optimizer(lr, max_norm).step(scaled)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norm = S.clip_grads_(grads, 0.5, out=scaled)
        again = a.step(scaled)
    rng = torch.Generator(device="cuda").manual_seed(112)
    for replay in range(4):
        say("replay", replay)
        lr.fill_(0.5 / (replay + 1))
        for g in grads:
            g.copy_(_values(rng, g.numel(), g.dtype, 0.02))
        graph.replay()
        torch.cuda.synchronize()
        out = [torch.empty_like(g) for g in grads]
        want = S.clip_grads_(grads, 0.5, out=out)
        want_again = b.step(out)
        assert torch.equal(norm, want) and (again is None) == (max_norm is None)
        assert again is None or torch.equal(again, want_again)
        assert a._step.tolist() == b._step.tolist() == [4 + replay, 0]
        for x, y in zip(net.state() + scaled, other.state() + out):
            assert torch.equal(x, y)


@pytest.mark.parametrize("sizes", LISTS)
def test_a_rate_on_the_device_is_the_hosts(sizes):
    net, other = (Several(KINDS["mixed"], LISTS[sizes]) for _ in range(2))
    lr = torch.tensor(0.25, device="cuda")  # exact in fp32
    a, b = net.optimizer(lr, 0.5), other.optimizer(0.25, 0.5)
    for rate in (0.25, 0.125):
        lr.fill_(rate)
        b.lr = rate
        a.step(net.grads)
        b.step(other.grads)
        for x, y in zip(net.state(), other.state()):
            assert torch.equal(x, y)
    assert a._step.tolist() == [5, 0]
