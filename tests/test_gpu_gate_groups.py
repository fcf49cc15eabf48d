"""Gates shared by rows, with as many groups as half the workgroups that fill
the GPU and more: gradients against the oracle, as their bounds are."""
import pytest
import torch

from gpu_util import say
from test_gpu_block_norm import BF16, F16, F32, make, run, verify

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("shape", [(128, 130, 64), (129, 130, 64), (129, 67, 200), (200, 40, 384),
                                   (255, 17, 500), (257, 70, 33), (600, 70, 64), (1000, 40, 64),
                                   (300, 30, 5), (129, 9, 2500)])
@pytest.mark.parametrize("types", [(F32, F32), (BF16, BF16), (F32, F16)])
def test_groups_around_the_number_of_workgroups(shape, types):
    say("groups", shape, types)
    gate = (shape[0], 1, shape[2])
    verify(make(shape, types, gate=gate, act="sigmoid", seed=100))
    verify(make(shape, types, gate=gate, act="none", weights=False, seed=101))


@pytest.mark.parametrize("shape", [(129, 130, 64), (1000, 40, 64)])
def test_the_gates_gradient_alone_and_left_out(shape):
    """The sums over a group are kept where they are asked for only."""
    t, dr, dh, act = make(shape, (F32, BF16), gate=(shape[0], 1, shape[2]), act="sigmoid", seed=102)
    every = run(t, dr, dh, act)[2]
    for leaf in ("gate", "scale", "x"):
        for k, v in t.items():
            v.requires_grad_(k == leaf)
        assert torch.equal(run(t, dr, dh, act, leaves=[leaf])[2][leaf], every[leaf]), leaf
