"""Attention at the ends of its range: scales that fp32 does not hold."""

import pytest
import torch

from block_oracle import Attention
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
