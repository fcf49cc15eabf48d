"""Clipping and AdamW, and what surrounds their launches."""
import pytest
import torch

import ssim_loss_amd as S
from test_gpu_train_update import F32, _list

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
