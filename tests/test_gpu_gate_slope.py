"""The gradient of a sigmoid gate that is almost open or almost closed: its
slope a (1 - a) keeps its bits where 1 - a is far below a's last one."""
import math

import pytest
import torch

from gpu_util import say
from test_gpu_block_norm import BF16, F16, F32, make, run
from train_oracle import U, Joint, activate, check, rounding

pytestmark = pytest.mark.gpu


def verify(made):
    t, dr, dh, act = made
    got = run(t, dr, dh, act)[2]["gate"]
    # The oracle forms 1 - a in 64 bits, which leaves nothing of it from g = 37 on;
    # here the gradient is that of the gate's value a, times the slope by itself.
    g = t["gate"].detach().cpu().double()
    a, far = activate(g, act), torch.exp(-g.abs())
    slope = far / (1 + far) ** 2
    of_value = Joint(*{**t, "gate": a}.values(), 1e-6, "none", dr, dh).grads["gate"][0]
    dg = of_value * slope
    # The oracle's bound takes a for the slope's magnitude.  Here it takes the
    # slope itself, plus what that may be off by: the exponential (its argument's
    # rounding in a half type's fast one), a twice, three products.
    half = t["branch"].dtype != F32
    wide, bound = Joint(*t.values(), 1e-6, act, dr, dh).grads["gate"]
    bound = (bound - rounding(wide, t["branch"].dtype) * 1.01) / a * slope
    act_u = 6.0 + (2.0 * g.abs() if half else 0.0)
    tight = bound + dg.abs() * (3 * act_u + 4) * U + rounding(dg, t["branch"].dtype) * 1.01
    check(got, dg, tight, "gradient of the gate")
    assert dg.any()


# a gate for each row; shared by few rows (uncut groups); by many (cut)
@pytest.mark.parametrize("shape,gate", [((6, 200), (6, 200)), ((6, 2000), (6, 2000)),
                                        ((4, 3000), (4, 3000)), ((2, 9000), (2, 9000)),
                                        ((6000, 2, 64), (6000, 1, 64)), ((2, 300, 200), (2, 1, 200)),
                                        ((2, 12, 9000), (2, 1, 9000))])
@pytest.mark.parametrize("types", [(F32, F32), (F16, F16), (BF16, BF16), (F32, BF16)])
def test_open_and_closed_gates(shape, gate, types):
    say("gates", shape, gate, types)
    t, dr, dh, act = make(shape, types, gate=gate, act="sigmoid", seed=80)
    # (upstream gradients that keep the gate's far from fp16's smallest)
    dr, dh = dr * 1e3, dh * 1e3
    g = t["gate"]
    with torch.no_grad():
        far = torch.linspace(8, 17, g.numel(), device="cuda").view(g.shape)
        g.copy_(torch.where(torch.arange(g.numel(), device="cuda").view(g.shape) % 2 == 0, far, -far))
    verify((t, dr, dh, act))


@pytest.mark.parametrize("types", [(F32, F32), (BF16, BF16)])
def test_a_gate_far_past_the_last_bit(types):
    """exp(-80) is a number of both types; the slope is as well."""
    t, dr, dh, act = make((3, 700), types, gate=(3, 700), act="sigmoid", seed=81)
    with torch.no_grad():
        t["gate"][0] = 80.0
        t["gate"][1] = -80.0
        t["gate"][2] = 30.0
    verify((t, dr, dh, act))
    with torch.no_grad():
        t["gate"][0] = math.inf
        t["gate"][1] = -math.inf
        t["gate"][2, 0] = math.nan
    got = run(t, dr, dh, act)[2]["gate"]
    assert not got[:2].any() and torch.isnan(got[2, 0])
