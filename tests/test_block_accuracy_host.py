"""That the limits of test_gpu_block_accuracy notice what they are for: mistakes of a
hundredth, planted in the definition (no GPU needed)."""
import math

import pytest
import torch

from test_gpu_block_accuracy import EPS, LIMIT


def numbers(*shape, seed, std=1.0, mean=0.0, dtype):
    t = torch.randn(shape, generator=torch.Generator().manual_seed(seed), dtype=torch.float64) * std + mean
    return t.to(dtype).double()


def gradients(q, k, v, d_out, delta_factor=1.0, o_type=None):
    """dq and dk of one head, the first query seeing one key and each later one more."""
    scale, (n, m) = q.shape[1] ** -0.5, (q.shape[0], k.shape[0])
    seen = torch.arange(m)[None] <= torch.arange(n)[:, None] + (m - n)
    p = torch.softmax(torch.where(seen, scale * q @ k.t(), -math.inf), 1)
    o = p @ v
    if o_type is not None:
        o = o.to(o_type).double()
    ds = p * (d_out @ v.t() - delta_factor * (d_out * o).sum(1, keepdim=True))
    return scale * ds @ k, scale * ds.t() @ q


def apart(a, b):
    return [float((x - y).norm() / y.norm()) for x, y in zip(a, b)]


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("n,m,dim", [(70, 90, 64), (200, 200, 128)])
def test_a_delta_two_hundredths_off(n, m, dim, dtype):
    t = [numbers(n, dim, seed=1, std=1.2, dtype=dtype), numbers(m, dim, seed=2, dtype=dtype),
         numbers(m, dim, seed=3, mean=0.2, dtype=dtype), numbers(n, dim, seed=4, std=0.1, dtype=dtype)]
    for off in apart(gradients(*t, delta_factor=1.02), gradients(*t)):
        assert off > LIMIT[dtype], off


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_an_output_rounded_before_its_delta(dtype):
    n, m, size, std = 33, 1024, 30.0, 0.3
    t = [numbers(n, 64, seed=5, std=0.36, dtype=dtype), numbers(m, 64, seed=6, std=std, dtype=dtype),
         numbers(m, 64, seed=7, std=std, mean=size, dtype=dtype), numbers(n, 64, seed=8, std=0.1, dtype=dtype)]
    limit = 1.5 * math.sqrt(2 + (size / std) ** 2 / m) * EPS[dtype]
    for off in apart(gradients(*t, o_type=dtype), gradients(*t)):
        assert off > 2 * limit, off
