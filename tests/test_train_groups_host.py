"""How many workgroups the joint's backward deals the rows of shared gates out
to, from the workspace that it asks for (no GPU needed)."""
import ctypes

import pytest

import ssim_loss_amd as S
from test_train_host import NormInputs


def workgroups(groups, gate_rows, width, dtype):
    """At least: each leaves at most three rows of fp32 sums."""
    given = NormInputs(x=0x100000, branch=0x200000, gate=0x300000, rows=groups * gate_rows, width=width,
                       gate_rows=gate_rows, eps=1e-6, x_dtype=dtype, branch_dtype=dtype)
    return S.train.lib().ssim_block_norm_workspace_bytes(ctypes.byref(given)) // (3 * 4 * width)


@pytest.mark.parametrize("dtype", [0, 1, 2])
@pytest.mark.parametrize("width", [64, 100, 384, 1000])
@pytest.mark.parametrize("groups", [120, 127, 128, 129, 200, 255, 256, 257, 500, 1000, 3000])
def test_a_call_with_many_groups_fills_half_the_gpu(groups, width, dtype):
    """1024 rows to a group: more rows than 256 compute units hold at once."""
    assert workgroups(groups, 1024, width, dtype) >= 120
