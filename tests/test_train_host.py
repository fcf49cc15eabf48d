"""Host-side checks of the training operators (no GPU needed): the library
exports what its header declares, refuses bad arguments with the documented
codes before any HIP call, and the binding refuses bad tensors.  And the
oracle's gradients against differences of its own joint."""
import ctypes
import math
import os
import re

import pytest
import torch

import ssim_loss_amd as S
from train_oracle import Joint, joint

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "ssim_loss_amd", "train", "include", "ssim_train_amd.h")

VP, I64, I32, F64 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_double


class ClipItem(ctypes.Structure):
    _fields_ = [("grad", VP), ("out", VP), ("n", I64), ("dtype", I32), ("reserved", I32)]


class AdamItem(ctypes.Structure):
    _fields_ = [("grad", VP), ("param", VP), ("exp_avg", VP), ("exp_avg_sq", VP), ("master", VP),
                ("n", I64), ("grad_dtype", I32), ("param_dtype", I32)]


class AdamOptions(ctypes.Structure):
    _fields_ = [(n, F64) for n in ("lr", "beta1", "beta2", "eps", "weight_decay", "max_norm")] \
        + [("lr_device", VP)]


class NormInputs(ctypes.Structure):
    _fields_ = [(n, VP) for n in ("x", "branch", "gate", "scale", "post_weight", "pre_weight")] \
        + [(n, I64) for n in ("rows", "width", "gate_rows")] + [("eps", F64)] \
        + [(n, I32) for n in ("x_dtype", "branch_dtype", "gate_act", "reserved")]


class NormGrads(ctypes.Structure):
    _fields_ = [(n, VP) for n in ("x", "branch", "gate", "scale", "post_weight", "pre_weight")]


def test_library_exports_every_declared_symbol():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b(ssim_[a-z_0-9]+)\s*\(", text))
    assert {"ssim_clip_grads", "ssim_grad_norm", "ssim_adamw_step", "ssim_block_norm_forward",
            "ssim_block_norm_backward"} <= names
    lib = S.train.lib()
    for n in names:
        assert hasattr(lib, n), n
    v = int(re.search(r"#define SSIM_TRAIN_ABI_VERSION (\d+)", text).group(1))
    assert S.train.abi_version() == v == S.train.ABI_VERSION
    for code in range(0, -11, -1):
        assert lib.ssim_train_strerror(code)
    assert b"unknown" in lib.ssim_train_strerror(-99)
    assert isinstance(S.TrainError(-5, "here"), S.SsimError) and S.TrainError(-5, "here").code == -5


def _clip(items=((0x10000, 0x20000, 64, 0),), max_norm=1.0, norm=0x1000, ws=0x100000, count=None,
          call="ssim_clip_grads"):
    array = (ClipItem * max(1, len(items)))(*[ClipItem(*it, 0) for it in items])
    count = len(items) if count is None else count
    lib = S.train.lib()
    if call == "ssim_grad_norm":
        return lib.ssim_grad_norm(array, count, norm, ws, None)
    return lib.ssim_clip_grads(array, count, max_norm, norm, ws, None)


def test_clip_argument_errors_return_before_any_hip_call():
    assert _clip(norm=None) == -1
    assert _clip(ws=None) == -1
    assert S.train.lib().ssim_clip_grads(None, 1, 1.0, 0x1000, 0x100000, None) == -1
    assert _clip([(None, 0x20000, 64, 0)]) == -1
    assert _clip([(0x10000, None, 64, 0)]) == -1
    assert _clip(count=-1) == -2
    assert _clip([(0x10000, 0x20000, -1, 0)]) == -2
    assert _clip([(0x10002, 0x20000, 64, 0)]) == -2      # fp32 at 2 bytes
    assert _clip([(0x10000, 0x20001, 64, 2)]) == -2      # bf16 at an odd byte
    assert _clip(norm=0x1002) == -2
    assert _clip(ws=0x100004) == -2
    assert _clip([(0x10000, 0x20000, 64, 3)]) == -8
    assert _clip([(0x10000, 0x20000, 1 << 62, 0)]) == -4
    assert _clip([(0x10000, 0x20000, 1 << 45, 2)] * 3) == -4
    for bad in (-1.0, math.nan, math.inf):
        assert _clip(max_norm=bad) == -10
    assert _clip([(0x10000, 0x10000 + 64, 64, 0)]) == -5           # out overlaps its grad in part
    assert _clip([(0x10000, 0x20000, 64, 0), (0x20000, 0x30000, 64, 0)]) == -5
    assert _clip([(0x10000, 0x10000, 64, 0), (0x10000, 0x10000, 64, 0)]) == -5  # the same tensor twice
    assert _clip(norm=0x20000 + 4) == -5
    assert _clip(ws=0x10000 + 8) == -5
    assert _clip(norm=0x100000 + 8) == -5
    assert _clip([(0x10000, None, 64, 7)], call="ssim_grad_norm") == -8
    assert _clip([(0x10000, None, 64, 0)], norm=0x10000, call="ssim_grad_norm") == -5


def _adam(it=None, step=0x800, norm=0x1000, ws=0x100000, count=1, **options):
    o = dict(lr=1e-3, beta1=0.9, beta2=0.99, eps=1e-8, weight_decay=0.1, max_norm=1.0, lr_device=None)
    o.update(options)
    base = dict(grad=0x10000, param=0x20000, exp_avg=0x30000, exp_avg_sq=0x40000, master=None, n=64,
                grad_dtype=0, param_dtype=0)
    base.update(it or {})
    return S.train.lib().ssim_adamw_step(ctypes.byref(AdamItem(**base)), count,
                                         ctypes.byref(AdamOptions(**o)), step, norm, ws, None)


def test_adamw_argument_errors_return_before_any_hip_call():
    for name in ("grad", "param", "exp_avg", "exp_avg_sq"):
        assert _adam({name: None}) == -1, name
    assert _adam(step=None) == -1
    assert _adam(ws=None) == -1
    assert _adam(norm=None) == -1                      # clipping needs it
    assert _adam(count=-1) == -2
    assert _adam({"n": -1}) == -2
    assert _adam({"exp_avg": 0x30002}) == -2
    assert _adam({"master": 0x50001}) == -2
    assert _adam(step=0x804) == -2
    assert _adam(lr_device=0x902) == -2
    assert _adam({"param_dtype": 3}) == -8
    assert _adam({"grad_dtype": 1}) == -8              # an fp16 gradient of an fp32 parameter
    assert _adam({"grad_dtype": 1, "param_dtype": 2}) == -8
    assert _adam({"n": 1 << 60}) == -4
    for bad in (dict(lr=-1.0), dict(lr=math.nan), dict(lr=math.inf), dict(beta1=1.0),
                dict(beta2=-0.1), dict(beta1=math.nan), dict(eps=-1e-9), dict(weight_decay=-0.1),
                dict(max_norm=-1.0), dict(max_norm=math.nan)):
        assert _adam(**bad) == -10, bad
    assert _adam({"exp_avg": 0x20000 + 128}) == -5     # inside the parameter
    assert _adam({"grad": 0x40000}) == -5
    assert _adam({"master": 0x20000}) == -5
    assert _adam(step=0x20000 + 8) == -5
    assert _adam(norm=0x30000) == -5
    assert _adam(lr_device=0x40000 + 4) == -5


def _inputs(**kw):
    base = dict(x=0x100000, branch=0x200000, gate=0x300000, scale=0x400000, post_weight=0x410000,
                pre_weight=0x420000, rows=8, width=64, gate_rows=1, eps=1e-6, x_dtype=0,
                branch_dtype=0, gate_act=0, reserved=0)
    base.update(kw)
    return ctypes.byref(NormInputs(**base))


def _fwd(residual=0x500000, normed=0x600000, stats=0x700000, **kw):
    return S.train.lib().ssim_block_norm_forward(_inputs(**kw), residual, normed, stats, None)


def _bwd(stats=0x700000, dr=0x800000, dh=0x900000, ws=0xA00000, grads=None, **kw):
    g = dict(x=0xB00000, branch=0xC00000, gate=0xD00000, scale=0xE00000, post_weight=0xE10000,
             pre_weight=0xE20000)
    g.update(grads or {})
    return S.train.lib().ssim_block_norm_backward(_inputs(**kw), stats, dr, dh,
                                                  ctypes.byref(NormGrads(**g)), ws, None)


@pytest.mark.parametrize("call", [_fwd, _bwd])
def test_block_norm_input_errors_return_before_any_hip_call(call):
    assert call(x=None) == -1
    assert call(branch=None) == -1
    assert call(rows=-1) == -2
    assert call(width=0) == -2
    assert call(width=16385) == -2
    assert call(gate_rows=0) == -2
    assert call(gate_rows=3) == -2                     # does not divide 8 rows
    assert call(x=0x100002) == -2
    assert call(scale=0x400002) == -2
    assert call(branch_dtype=1, x_dtype=2) == -8
    assert call(branch_dtype=0, x_dtype=1) == -8       # a half residual of fp32 blocks
    assert call(branch_dtype=5) == -8
    assert call(gate_act=2) == -10
    for bad in (-1e-6, math.nan, math.inf):
        assert call(eps=bad) == -10
    assert call(rows=1 << 50) == -4
    assert S.train.lib().ssim_block_norm_forward(None, 1, 1, 1, None) == -1


def test_block_norm_output_errors_return_before_any_hip_call():
    assert _fwd(residual=None) == -1
    assert _fwd(normed=None) == -1
    assert _fwd(residual=0x500002) == -2
    assert _fwd(residual=0x100000) == -5               # in place
    assert _fwd(normed=0x300000 + 64) == -5            # over the gate
    assert _fwd(stats=0x600000 + 8) == -5
    assert _fwd(rows=0, x=None, residual=None) == 0    # nothing to do: no launch
    assert _bwd(stats=None) == -1
    assert _bwd(ws=None) == -1
    assert _bwd(ws=0xA00008) == -2
    assert _bwd(gate=None) == -1                       # the gradient of a gate that is not there
    assert _bwd(scale=None) == -1
    assert _bwd(grads={"x": 0x800000}) == -5           # over the upstream gradient
    assert _bwd(grads={"scale": 0xE10000 + 16}) == -5
    assert _bwd(ws=0xC00000) == -5
    none = dict(x=None, branch=None, gate=None, scale=None, post_weight=None, pre_weight=None)
    assert _bwd(grads=none) == 0                       # nothing to do: no launch


def test_block_norm_workspace_bytes():
    f = lambda **kw: S.train.lib().ssim_block_norm_workspace_bytes(_inputs(**kw))
    assert f(rows=0) == 0 and f(width=0) == 0 and f(branch_dtype=9) == 0
    assert f() >= 2 * 4 * 64
    assert f() % 16 == 0 and f(width=33) % 16 == 0
    # it stays a small share of a large call's own traffic
    assert f(rows=1 << 20, width=4096) < 64 << 20
    assert f(rows=1 << 20, width=4096, gate_rows=1 << 18) < 64 << 20


def test_binding_refuses_what_is_not_a_gpu_tensor_of_a_known_type():
    t = torch.ones(4)
    for call in (lambda: S.clip_grads_([t], 1.0), lambda: S.grad_norm([t]),
                 lambda: S.clip_grads_(t, 1.0), lambda: S.clip_grads_([1.0], 1.0),
                 lambda: S.block_norm(t, t), lambda: S.block_norm(1, t),
                 lambda: S.AdamW([t]), lambda: S.AdamW([3])):
        with pytest.raises(TypeError):
            call()
    for call in (lambda: S.clip_grads_([], 1.0), lambda: S.AdamW([]),
                 lambda: S.clip_grads_([t], math.nan), lambda: S.clip_grads_([t], -1.0),
                 lambda: S.clip_grads_([t], 1.0, out=[]),
                 lambda: S.block_norm(t, t, gate_act="tanh")):
        with pytest.raises(ValueError):
            call()


@pytest.mark.parametrize("act", ["none", "sigmoid"])
@pytest.mark.parametrize("gate_shape", [(2, 3, 7), (2, 1, 7), (1, 1, 7)])
def test_oracle_gradients_are_the_joints_differences(gate_shape, act):
    g = torch.Generator().manual_seed(3)
    n = lambda *s: torch.randn(s, generator=g, dtype=torch.float64)
    t = {"x": n(2, 3, 7), "branch": n(2, 3, 7), "gate": n(*gate_shape), "scale": n(7),
         "post_weight": n(7), "pre_weight": n(7)}
    dr, dh = n(2, 3, 7), n(2, 3, 7)
    f = lambda v: sum((o * d).sum() for o, d in zip(joint(*v.values(), 1e-6, act), (dr, dh)))
    # (the oracle takes types for its bounds only; the values stay 64-bit)
    want = Joint(*[v.float() for v in t.values()], 1e-6, act, dr.float(), dh.float()).grads
    t = {k: v.float().double() for k, v in t.items()}
    dr, dh = dr.float().double(), dh.float().double()
    step = 1e-5
    for name, v in t.items():
        along = n(*v.shape)
        up, down = ({**t, name: v + s * along} for s in (step, -step))
        slope = (f(up) - f(down)) / (2 * step)
        assert abs(slope - (want[name][0] * along).sum()) < 1e-7 * (1 + abs(slope)), name
