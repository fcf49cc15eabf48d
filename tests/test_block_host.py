"""Host-side checks of the operators inside a block (no GPU needed): the C entry
points refuse bad arguments with the documented codes before any HIP call,
workspaces have the sizes that their calls use, the binding refuses bad tensors
and what goes past torch's dispatcher; and the oracle's gradients against
differences of its own definitions."""
import ctypes
import math

import pytest
import torch
import torch.autograd.forward_ad as forward_ad
from torch.fx.experimental.proxy_tensor import make_fx

import ssim_loss_amd as S
from block_oracle import Attention, Gated, rotary
from train_oracle import TINY

VP, I64, I32, F64 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_double


class RotaryInputs(ctypes.Structure):
    _fields_ = [(n, VP) for n in ("q", "k", "positions")] \
        + [("q_stride", I64 * 3), ("k_stride", I64 * 3), ("position_stride", I64 * 2), ("batch", I64), ("tokens", I64)] \
        + [(n, I32) for n in ("q_heads", "k_heads", "dim", "axes")] + [("axis_size", I32 * 4)] \
        + [(n, I32) for n in ("pairs", "position_type", "dtype", "inverse")] + [("base", F64)]


class AttentionInputs(ctypes.Structure):
    _fields_ = [(n, VP) for n in ("q", "k", "v", "q_lengths", "k_lengths")] \
        + [(n, I64 * 3) for n in ("q_stride", "k_stride", "v_stride")] + [(n, I64) for n in ("batch", "q_tokens", "k_tokens")] \
        + [(n, I32) for n in ("heads", "kv_heads", "dim", "causal", "dtype", "reserved")] + [("scale", F64)]


class GatedInputs(ctypes.Structure):
    _fields_ = [(n, VP) for n in ("x", "w_gate", "w_up", "b_gate", "b_up")] + [(n, I64) for n in ("rows", "width", "hidden")] \
        + [(n, I32) for n in ("act", "dtype")]


class GatedGrads(ctypes.Structure):
    _fields_ = [(n, VP) for n in ("x", "w_gate", "w_up", "b_gate", "b_up")]


F32, F16, BF16 = 0, 1, 2
M = 1 << 20  # the tensors' made-up addresses are this far apart


def strides(tokens, heads, dim):
    return (I64 * 3)(tokens * heads * dim, heads * dim, dim)


def rotary_inputs(**kw):
    base = dict(q=M, k=2 * M, positions=3 * M, q_stride=strides(5, 4, 32), k_stride=strides(5, 2, 32),
                position_stride=(I64 * 2)(0, 2), batch=2, tokens=5, q_heads=4, k_heads=2, dim=32, axes=2,
                axis_size=(I32 * 4)(8, 16), pairs=0, position_type=0, dtype=BF16, inverse=0, base=1e4)
    base.update(kw)
    return RotaryInputs(**base)


def rot(q_out=4 * M, k_out=5 * M, **kw):
    return S.train.lib().ssim_rotary(ctypes.byref(rotary_inputs(**kw)), q_out, k_out, None)


def test_rotary_argument_errors_return_before_any_hip_call():
    for name in ("q", "positions"):
        assert rot(**{name: None}) == -1, name
    assert rot(q_out=None) == -1 and rot(k_out=None) == -1
    assert S.train.lib().ssim_rotary(None, M, M, None) == -1
    for bad in (dict(batch=-1), dict(tokens=-1), dict(dim=0), dict(dim=513), dict(q_heads=0), dict(k_heads=0), dict(axes=0),
                dict(axes=5), dict(axis_size=(I32 * 4)(7, 8)), dict(axis_size=(I32 * 4)(0, 8)),
                dict(axis_size=(I32 * 4)(20, 16)), dict(q=M + 1), dict(positions=M * 3 + 2), dict(q_stride=(I64 * 3)(1, -1, 1))):
        assert rot(**bad) == -2, bad
    assert rot(q_out=4 * M + 1) == -2
    assert rot(dtype=3) == -8 and rot(position_type=3) == -8
    for bad in (dict(pairs=2), dict(inverse=2), dict(base=0.0), dict(base=-1.0), dict(base=math.nan), dict(base=math.inf)):
        assert rot(**bad) == -10, bad
    assert rot(tokens=1 << 45) == -4
    far = (I64 * 3)(1 << 46, 1 << 46, 1)
    assert rot(batch=1 << 20, q_stride=far) == -4 and rot(tokens=1 << 20, k_stride=far) == -4  # past 64 bits in bytes
    assert rot(batch=1 << 20, position_stride=(I64 * 2)(1 << 46, 1)) == -4
    assert rot(q_out=M + 64) == -5 and rot(q_out=5 * M) == -5 and rot(k_out=3 * M) == -5
    assert rot(batch=0, q=None) == 0 and rot(tokens=0, q_out=None) == 0
    assert rot(k=None, k_out=None, q_out=M) == -5  # in place


def attention_inputs(dtype=BF16, **kw):
    base = dict(q=M, k=2 * M, v=3 * M, q_lengths=4 * M, k_lengths=None, q_stride=strides(5, 4, 32), k_stride=strides(7, 2, 32),
                v_stride=strides(7, 2, 32), batch=2, q_tokens=5, k_tokens=7, heads=4, kv_heads=2, dim=32, causal=1,
                dtype=dtype, reserved=0, scale=0.5)
    base.update(kw)
    return AttentionInputs(**base)


def att(out=5 * M, lse=6 * M, rest=7 * M, ws=8 * M, **kw):
    return S.train.lib().ssim_attention_forward(ctypes.byref(attention_inputs(**kw)), out, lse, rest, ws, None)


def att_back(out=5 * M, lse=6 * M, rest=7 * M, d_out=9 * M, dq=10 * M, dk=11 * M, dv=12 * M, ws=8 * M, **kw):
    return S.train.lib().ssim_attention_backward(ctypes.byref(attention_inputs(**kw)), out, lse, rest, d_out, dq, dk, dv, ws, None)


@pytest.mark.parametrize("call", [att, att_back])
def test_attention_input_errors_return_before_any_hip_call(call):
    for name in ("q", "k", "v"):
        assert call(**{name: None}) == -1, name
    for bad in (dict(batch=-1), dict(q_tokens=-1), dict(k_tokens=1 << 24), dict(heads=0), dict(kv_heads=3), dict(dim=0),
                dict(dim=12), dict(dim=136), dict(q=M + 8), dict(k=2 * M + 2), dict(q_lengths=4 * M + 2),
                dict(q_stride=(I64 * 3)(640, 128, 30)), dict(k_stride=(I64 * 3)(448, 24, 32)),
                dict(v_stride=(I64 * 3)(448, -64, 32)), dict(v_stride=(I64 * 3)(1 << 30, 1 << 24, 32))):
        assert call(**bad) == -2, bad
    assert call(dtype=5) == -8
    for bad in (dict(scale=0.0), dict(scale=-1.0), dict(scale=math.nan), dict(scale=1e300), dict(causal=2)):
        assert call(**bad) == -10, bad
    assert call(batch=1 << 30) == -4
    assert call(batch=1 << 20, kv_heads=1, q_stride=(I64 * 3)(1 << 44, 128, 32)) == -4  # past 64 bits in bytes
    assert call(batch=1 << 24, q_tokens=(1 << 24) - 1, heads=65536, kv_heads=1) == -4
    assert call(q_tokens=(1 << 24) - 1, heads=128, kv_heads=1, dim=8, batch=1, q_stride=(I64 * 3)(0, 1024, 8)) == -4  # 2^31 rows
    assert call(batch=0, q=None) == 0
    assert S.train.lib().ssim_attention_forward(None, M, M, M, M, None) == -1


def test_attention_output_errors_return_before_any_hip_call():
    assert att(out=None) == -1
    assert att(out=5 * M + 1) == -2 and att(lse=6 * M + 2) == -2
    assert att(out=M + 64) == -5 and att(lse=5 * M) == -5 and att(rest=5 * M) == -5 and att(out=4 * M) == -5
    assert att(q_tokens=0, out=None) == 0
    for name in ("out", "lse", "rest", "d_out", "ws"):
        assert att_back(**{name: None}) == -1, name
    assert att_back(dtype=F32, rest=None, dq=11 * M, dk=11 * M) == -5  # fp32 needs no rest
    assert att_back(d_out=9 * M + 8) == -2 and att_back(rest=7 * M + 2) == -2 and att_back(ws=8 * M + 4) == -2
    assert att_back(dq=9 * M) == -5 and att_back(dk=12 * M + 16) == -5 and att_back(ws=5 * M) == -5
    assert att_back(dq=None, dk=None, dv=None) == 0
    assert att_back(q_tokens=0, k_tokens=0) == 0


def test_attention_workspaces():
    lib = S.train.lib()
    f = lambda **kw: lib.ssim_attention_workspace_bytes(ctypes.byref(attention_inputs(**kw)))
    b = lambda **kw: lib.ssim_attention_backward_workspace_bytes(ctypes.byref(attention_inputs(**kw)))
    assert f() == 0  # few keys: one part
    few = dict(q_tokens=1, k_tokens=100000)
    assert f(**few) > 0 and f(**few) % 16 == 0
    assert f(q_tokens=4096, k_tokens=4096, batch=64) == 0
    assert b() == 2 * 4 * 5 * 4 and b(dtype=F16) == 2 * 4 * 5 * 4 + 2 * 2 * 16 * 8 and b(dim=7) == 0
    assert att(ws=None) != -1 and att(ws=None, k_stride=strides(1000, 2, 32), **few) == -1


def gated_inputs(**kw):
    base = dict(x=16 * M, w_gate=32 * M, w_up=48 * M, b_gate=64 * M, b_up=65 * M, rows=100, width=64, hidden=96, act=0, dtype=BF16)
    base.update(kw)
    return GatedInputs(**base)


def gat(out=80 * M, g=96 * M, u=112 * M, ws=128 * M, **kw):
    return S.train.lib().ssim_gated_linear_forward(ctypes.byref(gated_inputs(**kw)), out, g, u, ws, None)


def gat_back(g=96 * M, u=112 * M, d_out=80 * M, ws=128 * M, grads=None, **kw):
    wanted = dict(x=144 * M, w_gate=160 * M, w_up=176 * M, b_gate=192 * M, b_up=193 * M)
    wanted.update(grads or {})
    return S.train.lib().ssim_gated_linear_backward(ctypes.byref(gated_inputs(**kw)), g, u, d_out,
                                                    ctypes.byref(GatedGrads(**wanted)), ws, None)


@pytest.mark.parametrize("call", [gat, gat_back])
def test_gated_linear_input_errors_return_before_any_hip_call(call):
    for name in ("x", "w_gate", "w_up"):
        assert call(**{name: None}) == -1, name
    for bad in (dict(rows=-1), dict(width=0), dict(hidden=0), dict(width=(1 << 20) + 1), dict(x=16 * M + 1)):
        assert call(**bad) == -2, bad
    assert call(g=96 * M + 8) == -2
    assert call(dtype=7) == -8 and call(act=3) == -10 and call(act=-1) == -10
    assert call(rows=1 << 29) == -4
    assert call(width=63, ws=None) == -1  # rows that have to be copied


def test_gated_linear_output_errors_return_before_any_hip_call():
    assert gat(out=None) == -1 and gat(u=None) == -1
    assert gat(out=16 * M + 64) == -5 and gat(g=80 * M) == -5 and gat(out=32 * M) == -5
    assert gat(rows=0, out=None) == 0
    for name in ("g", "u", "d_out", "ws"):
        assert gat_back(**{name: None}) == -1, name
    assert gat_back(b_gate=None) == -1  # the gradient of a bias that is not there
    assert gat_back(grads=dict(x=80 * M)) == -5 and gat_back(grads=dict(w_up=160 * M)) == -5 and gat_back(ws=144 * M) == -5
    none = dict(x=None, w_gate=None, w_up=None, b_gate=None, b_up=None)
    assert gat_back(grads=none) == 0
    assert S.train.lib().ssim_gated_linear_backward(ctypes.byref(gated_inputs()), 1, 1, 1, None, 1, None) == -1


def test_gated_linear_sizes():
    lib = S.train.lib()
    f = lambda **kw: lib.ssim_gated_linear_workspace_bytes(ctypes.byref(gated_inputs(**kw)))
    b = lambda **kw: lib.ssim_gated_linear_backward_workspace_bytes(ctypes.byref(gated_inputs(**kw)))
    n = lambda **kw: lib.ssim_gated_linear_saved_elements(ctypes.byref(gated_inputs(**kw)))
    assert f() == 0 and f(width=63) == (100 + 2 * 96) * 64 * 2 and f(x=16 * M + 2) == (100 + 2 * 96) * 64 * 2
    assert f(width=63, rows=8) == 0  # few rows are read where they lie
    assert n() == 100 * 96 and n(hidden=97) == 100 * 104 and n(hidden=97, dtype=F32) == 100 * 100 and n(width=0) == 0
    assert b() >= 2 * 100 * 96 * 2 and b(hidden=97) % 16 == 0 and b(act=9) == 0
    # parts of products stay within a few times the result
    assert b(rows=64, width=64, hidden=1 << 16) < 64 * (1 << 16) * 4 * 4 + 20 * 2 * 64 * (1 << 16) * 4


# ------------------------------------------------------------------ the binding
def calls(t):
    """Each entry point on the tensor t, in each place."""
    a, w, p = torch.ones(1, 2, 2, 8), torch.ones(4, 8), torch.zeros(2, 1)
    r4 = lambda: t.reshape(1, 2, 2, 8)
    return {"rotary q": lambda: S.rotary(r4(), None, p, (8,)), "rotary k": lambda: S.rotary(a, r4(), p, (8,)),
            "rotary positions": lambda: S.rotary(a, None, t.reshape(-1)[:2].reshape(2, 1), (8,)),
            "attention q": lambda: S.attention(r4(), a, a), "attention k": lambda: S.attention(a, r4(), a),
            "attention v": lambda: S.attention(a, a, r4()), "gated x": lambda: S.gated_linear(t.reshape(4, 8), w, w),
            "gated w": lambda: S.gated_linear(w, w, t.reshape(4, 8)), "gated b": lambda: S.gated_linear(w, w, w, t.reshape(-1)[:4])}


NAMES = list(calls(torch.ones(4, 8)))


def test_binding_refuses_what_is_not_a_gpu_tensor_of_a_known_type():
    for name, call in calls(torch.ones(4, 8)).items():
        with pytest.raises(TypeError, match="GPU tensor"):
            call()
    for call in (lambda: S.rotary(1, None, 1, (8,)), lambda: S.attention(None, None, None), lambda: S.gated_linear(2.0, 1, 1)):
        with pytest.raises(TypeError):
            call()
    t = torch.ones(1, 2, 2, 8)
    for call in (lambda: S.rotary(t, None, t, (8,), pairs="both"), lambda: S.gated_linear(t, t, t, act="relu")):
        with pytest.raises(ValueError):
            call()


@pytest.mark.parametrize("which", NAMES)
def test_tensors_with_a_forward_mode_tangent_are_refused(which):
    with forward_ad.dual_level():
        dual = forward_ad.make_dual(torch.ones(4, 8), torch.full((4, 8), 2.0))
        with pytest.raises(NotImplementedError, match="forward-mode"):
            calls(dual)[which]()
        with pytest.raises(TypeError, match="GPU tensor"):
            calls(torch.ones(4, 8))[which]()


@pytest.mark.parametrize("which", NAMES)
def test_views_with_the_sign_turned_are_refused(which):
    with pytest.raises(NotImplementedError, match="sign"):
        calls(torch._neg_view(torch.ones(4, 8)))[which]()


@pytest.mark.parametrize("which", ["rotary q", "attention q", "gated x"])
@pytest.mark.parametrize("trace", [lambda f, x: torch.jit.trace(f, (x,)), lambda f, x: make_fx(f)(x)], ids=["jit", "fx"])
def test_tracers_are_refused(trace, which):
    def traced(t):
        out = t * 2.0
        calls(t)[which]()
        return out

    with pytest.raises(NotImplementedError, match="tracer"):
        trace(traced, torch.ones(4, 8))


# ------------------------------------------------------------------ the oracle
def slopes(f, leaves, grads):
    """Differences of f along a direction for each leaf, against its gradient."""
    rng = torch.Generator().manual_seed(5)
    for name, v in leaves.items():
        along = torch.randn(v.shape, generator=rng, dtype=torch.float64)
        up, down = ({**leaves, name: v + s * along} for s in (1e-5, -1e-5))
        slope = (f(up) - f(down)) / 2e-5
        assert abs(slope - float((grads[name] * along).sum())) < 1e-7 * (1 + abs(slope)), name


def numbers(*shape, seed=0):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed), dtype=torch.float64).float()


@pytest.fixture(autouse=True)
def tiny_of_64_bits(monkeypatch):
    monkeypatch.setitem(TINY, torch.float64, 0.0)


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("lengths", [None, (5, 3)])
def test_oracle_gradients_of_attention_are_differences(lengths, causal):
    t = {"q": numbers(2, 5, 4, 8, seed=1), "k": numbers(2, 6, 2, 8, seed=2), "v": numbers(2, 6, 2, 8, seed=3)}
    d_out = numbers(2, 5, 4, 8, seed=4)
    kw = dict(causal=causal, key_lengths=lengths)
    want = Attention(**t, d_out=d_out, **kw).value
    f = lambda v: float((Attention(**v, **kw).value["out"] * d_out.double()).sum())
    slopes(f, {k: v.double() for k, v in t.items()}, want)


@pytest.mark.parametrize("act", ["silu", "gelu", "sigmoid"])
def test_oracle_gradients_of_the_gated_layer_are_differences(act):
    t = {"x": numbers(3, 7, seed=1), "w_gate": numbers(5, 7, seed=2), "w_up": numbers(5, 7, seed=3), "b_gate": numbers(5, seed=4),
         "b_up": numbers(5, seed=5)}
    d_out = numbers(3, 5, seed=6)
    want = Gated(**t, act=act, d_out=d_out).value
    f = lambda v: float((Gated(**v, act=act).value["out"] * d_out.double()).sum())
    slopes(f, {k: v.double() for k, v in t.items()}, want)


@pytest.mark.parametrize("pairs", ["adjacent", "halves"])
def test_oracle_of_rotary_turns_back_and_keeps_lengths(pairs):
    x, p = numbers(2, 5, 3, 20), numbers(5, 2, seed=9) * 30
    y, _ = rotary(x, p, (6, 12), 100.0, pairs)
    back, _ = rotary(y, p, (6, 12), 100.0, pairs, -1.0)
    assert (back - x.double()).abs().max() < 1e-12
    assert torch.allclose(y.square().sum(-1), x.double().square().sum(-1))
    assert torch.equal(y[..., 18:], x.double()[..., 18:])
    # the scores of turned queries and keys depend on the distance alone
    q, k = numbers(1, 1, 1, 20, seed=1), numbers(1, 1, 1, 20, seed=2)
    at = lambda a, b: float((rotary(q, torch.tensor([a]), (6, 12), 100.0, pairs)[0]
                             * rotary(k, torch.tensor([b]), (6, 12), 100.0, pairs)[0]).sum())
    assert abs(at([3.0, 7.0], [1.0, 2.5]) - at([13.0, 4.0], [11.0, -0.5])) < 1e-12
