"""The rest of a training step around the SSIM loss, on AMD MI355X: the global
gradient norm and clipping by it, AdamW with the clipping fused in, the joint
between two blocks of an image network, and what lies inside a block: rotary
positions, attention and the gated layer, all with their gradients.

The C ABI is ``include/ssim_train_amd.h``; ``_bind`` (csrc/bind*.cpp) calls it on
torch tensors, on torch's current stream of their device.  The computation runs
in the HIP kernels of ``libssim_train_amd.so``; there is no fallback path.

  clip_grads_(grads, max_norm, out=None)  -> the gradients' global norm
  grad_norm(grads)                        -> the norm alone
  AdamW(params, ...).step(grads=None)     -> the norm before clipping, or None
  block_norm(x, branch, gate=..., ...)    -> (residual, normed), with autograd
  rotary(q, k, positions, axes, ...)      -> (q, k) turned, with autograd
  attention(q, k, v, ...)                 -> the attended values, with autograd
  gated_linear(x, w_gate, w_up, ...)      -> act(x w_gate^T) x w_up^T, with autograd
"""
from __future__ import annotations

import ctypes
import os
import threading

from .. import SsimError
from ..build import BIND_PATH, TRAIN_LIB_PATH

# SSIM_TRAIN_ABI_VERSION of include/ssim_train_amd.h that this package follows
ABI_VERSION = 2

GATE_ACT = {"none": 0, "sigmoid": 1}
PAIRS = {"adjacent": 0, "halves": 1}
GATED_ACT = {"silu": 0, "gelu": 1, "sigmoid": 2}

_lock = threading.Lock()
_lib = None
_module = None


class TrainError(SsimError):
    """A call of the training library returned an error code."""

    def __init__(self, code: int, where: str):
        text = lib().ssim_train_strerror(int(code)).decode()
        RuntimeError.__init__(self, f"{where}: {text} (code {code})")
        self.code = code


def _missing(path: str) -> ImportError:
    return ImportError(f"{path} is missing: build it first (python -m ssim_loss_amd.build or "
                       "__graft_entry__.build()); there is no fallback implementation")


def lib() -> ctypes.CDLL:
    """The C-ABI library, for callers of the C functions.  SSIM_TRAIN_AMD_LIB
    names another build of the same sources for them; the operators on tensors
    run in the one that their binding was linked with."""
    global _lib
    with _lock:
        if _lib is None:
            path = os.environ.get("SSIM_TRAIN_AMD_LIB", TRAIN_LIB_PATH)
            if not os.path.exists(path):
                raise _missing(path)
            L = ctypes.CDLL(path)
            i64, i32, vp, sz, f64 = (ctypes.c_int64, ctypes.c_int, ctypes.c_void_p,
                                     ctypes.c_size_t, ctypes.c_double)
            for name, result, args in (
                    ("ssim_train_abi_version", i32, []),
                    ("ssim_train_strerror", ctypes.c_char_p, [i32]),
                    ("ssim_update_workspace_bytes", sz, []),
                    ("ssim_clip_grads", i32, [vp, i64, f64, vp, vp, vp]),
                    ("ssim_grad_norm", i32, [vp, i64, vp, vp, vp]),
                    ("ssim_adamw_step", i32, [vp, i64, vp, vp, vp, vp, vp]),
                    ("ssim_block_norm_forward", i32, [vp, vp, vp, vp, vp]),
                    ("ssim_block_norm_workspace_bytes", sz, [vp]),
                    ("ssim_block_norm_backward", i32, [vp, vp, vp, vp, vp, vp, vp]),
                    ("ssim_rotary", i32, [vp, vp, vp, vp]),
                    ("ssim_attention_workspace_bytes", sz, [vp]),
                    ("ssim_attention_forward", i32, [vp, vp, vp, vp, vp, vp]),
                    ("ssim_attention_backward_workspace_bytes", sz, [vp]),
                    ("ssim_attention_backward", i32, [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp]),
                    ("ssim_gated_linear_saved_elements", sz, [vp]),
                    ("ssim_gated_linear_workspace_bytes", sz, [vp]),
                    ("ssim_gated_linear_backward_workspace_bytes", sz, [vp]),
                    ("ssim_gated_linear_forward", i32, [vp, vp, vp, vp, vp, vp]),
                    ("ssim_gated_linear_backward", i32, [vp, vp, vp, vp, vp, vp, vp])):
                function = getattr(L, name)
                function.restype = result
                function.argtypes = args
            if L.ssim_train_abi_version() != ABI_VERSION:
                raise ImportError(
                    f"{path} implements ABI version {L.ssim_train_abi_version()}, this package "
                    f"version {ABI_VERSION}: rebuild it")
            _lib = L
    return _lib


def abi_version() -> int:
    return int(lib().ssim_train_abi_version())


def _native():
    global _module
    if _module is None:
        if not os.path.exists(BIND_PATH):
            raise _missing(BIND_PATH)
        import torch  # noqa: F401  (its libraries first)

        from . import _bind as module

        _module = module
    return _module


# --------------------------------------------------------------------------- clipping
def clip_grads_(grads, max_norm, out=None):
    """Scales `grads`, a list of GPU tensors (float32, float16, bfloat16, mixed as
    they come; contiguous, or channels_last or another permutation of it), by c = min(1, max_norm / (norm + 1e-6)),
    where norm is the root of the sum of all their squares, formed in fp64.

    Returns the norm before clipping, a 0-d float32 tensor; nothing waits for
    it.  Writes to `out` (tensors of the same shapes, strides and types) if given,
    else in place.  A NaN or infinite gradient makes the norm so, and the outputs
    follow the formula.  A tensor may be in the list once."""
    return _native().clip_grads(grads, max_norm, out)


def grad_norm(grads):
    """The global norm that clip_grads_ returns, without scaling."""
    return _native().grad_norm(grads)


# --------------------------------------------------------------------------- AdamW
class AdamW:
    """AdamW over a list of parameters, with clipping by the gradients' global
    norm in the same pass:

        g' = min(1, max_norm / (norm + 1e-6)) g
        m  = beta1 m + (1 - beta1) g'          v = beta2 v + (1 - beta2) g'^2
        w  = (1 - lr weight_decay) w - lr (m / (1 - beta1^t)) / (sqrt(v / (1 - beta2^t)) + eps)

    params:  GPU tensors of float32, float16 or bfloat16, contiguous or a
             permutation of it such as channels_last; gradients and states have
             their parameter's strides.
    lr:      a number, which may be changed between steps, or one float32 on
             the parameters' device: a captured graph then follows its value.
    max_norm: None: no clipping, and no norm is formed.
    exp_avgs, exp_avg_sqs: m and v to go on from, float32 (default: zeros).
    masters: float32 weights, one for each parameter (None entries: the
             parameter holds the weights), of which the parameters receive
             rounded copies.  Without one a half-type parameter is updated in
             float32 and rounded to its type, and updates below half a step of
             that type are lost.
    step:    updates done before.

    The number of updates is kept on the device, so a captured step may be
    replayed.  It is one number for all parameters."""

    def __init__(self, params, lr=1e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=1e-2,
                 max_norm=None, exp_avgs=None, exp_avg_sqs=None, masters=None, step=0):
        import torch

        self.params = list(params)
        if not self.params:
            raise ValueError("params must hold at least one tensor")
        for k, p in enumerate(self.params):
            if not isinstance(p, torch.Tensor):
                raise TypeError(f"params[{k}] must be a torch.Tensor")
            if p.device.type != "cuda":
                raise TypeError(f"params[{k}] must be a GPU tensor, got device {p.device}")
        self.lr = lr
        self.betas = (float(betas[0]), float(betas[1]))
        self.eps = float(eps)
        self.weight_decay = float(weight_decay)
        self.max_norm = None if max_norm is None else float(max_norm)
        if not isinstance(lr, torch.Tensor) and not 0.0 <= lr < float("inf"):
            raise ValueError("lr must be a number >= 0")
        if not all(0.0 <= b < 1.0 for b in self.betas):
            raise ValueError("betas must lie in [0, 1)")
        if not (0.0 <= self.eps < float("inf") and 0.0 <= self.weight_decay < float("inf")):
            raise ValueError("eps and weight_decay must be numbers >= 0")
        if self.max_norm is not None and not 0.0 <= self.max_norm < float("inf"):
            raise ValueError("max_norm must be a number >= 0, or None")
        if int(step) < 0:
            raise ValueError("step must be >= 0")

        def states(given):
            if given is not None:
                return list(given)
            return [torch.zeros_like(p, dtype=torch.float32)
                    for p in self.params]

        with torch.no_grad():
            self.exp_avgs = states(exp_avgs)
            self.exp_avg_sqs = states(exp_avg_sqs)
            self.masters = None if masters is None else list(masters)
            # (the second word is the library's, 0 between calls)
            self._step = torch.tensor([int(step), 0], dtype=torch.int64,
                                      device=self.params[0].device)
        for name in ("exp_avgs", "exp_avg_sqs", "masters"):
            held = getattr(self, name)
            if held is not None and len(held) != len(self.params):
                raise ValueError(f"{name} must have as many tensors as params")

    def step(self, grads=None):
        """One update from `grads` (default: each parameter's .grad; a None
        entry leaves its parameter and state as they are).  Returns the
        gradients' norm before clipping, a 0-d float32 tensor (None without
        clipping); nothing waits for it."""
        if grads is None:
            grads = [p.grad for p in self.params]
        return _native().adamw_step(grads, self.params, self.exp_avgs, self.exp_avg_sqs,
                                  self.masters, self._step, self.lr, self.betas[0], self.betas[1],
                                  self.eps, self.weight_decay, self.max_norm)

    def zero_grad(self) -> None:
        for p in self.params:
            p.grad = None

    @property
    def steps(self) -> int:
        """Updates done (waits for the device)."""
        return int(self._step[0].item())

    def state_dict(self) -> dict:
        """Copies of the state: exp_avgs, exp_avg_sqs, masters, step (waits
        for the device)."""
        def copies(held):
            return None if held is None else [None if t is None else t.detach().clone()
                                              for t in held]

        return {"exp_avgs": copies(self.exp_avgs), "exp_avg_sqs": copies(self.exp_avg_sqs),
                "masters": copies(self.masters), "step": self.steps}

    def load_state_dict(self, state: dict) -> None:
        """Copies a state_dict's values into this optimizer's tensors.  It must
        have been taken from parameters of the same shapes, with masters for
        the same ones."""
        import torch

        pairs = []
        for name in ("exp_avgs", "exp_avg_sqs", "masters"):
            held, given = getattr(self, name) or [], state[name] or []
            if len(held) != len(given):
                raise ValueError(f"{name}: {len(given)} tensors for {len(held)}")
            for k, (to, by) in enumerate(zip(held, given)):
                if (to is None) != (by is None) or (to is not None and to.shape != by.shape):
                    raise ValueError(f"{name}[{k}] does not have its parameter's shape")
                if to is not None:
                    pairs.append((to, by))
        with torch.no_grad():
            for to, by in pairs:
                to.copy_(by)
            self._step[0].fill_(int(state["step"]))


# --------------------------------------------------------------------------- the joint of two blocks
def block_norm(x, branch, gate=None, scale=None, post_weight=None, pre_weight=None, eps=1e-6,
               gate_act="none"):
    """The joint between two blocks of a network, in one pass over each row:

        residual = x + act(gate) * scale * post_weight * branch / rms(branch)
        normed   = residual / rms(residual) * pre_weight
        rms(v)   = sqrt(mean(v^2 over the last dimension) + eps)

    x:       [..., width], the residual stream: branch's type, or float32.
    branch:  [..., width], the block's output: float32, float16 or bfloat16.
    gate:    branch's type; x's shape (a gate for each token), or with ones in
             the place of the last few dimensions before the width (e.g.
             [batch, 1, width]: one for each sample); None: 1.
    scale, post_weight, pre_weight: float32 [width]; None: 1.
    gate_act: "none" or "sigmoid".

    Returns (residual, normed) of x's and branch's types; arithmetic is
    float32, and normed is formed from the residual before its rounding.
    Gradients of all tensor inputs are available, gradients of gradients and
    forward-mode derivatives are not.  Tensors must be contiguous; the width is at most 16384."""
    act = GATE_ACT.get(gate_act)
    if act is None:
        raise ValueError(f"gate_act must be 'none' or 'sigmoid', got {gate_act!r}")
    return _native().block_norm(x, branch, gate, scale, post_weight, pre_weight, eps, act)


# --------------------------------------------------------------------------- inside a block
def rotary(q, k, positions, axes, base=10000.0, pairs="adjacent"):
    """Queries and keys turned by their positions along several axes, such as
    (time, height, width), in one launch.

    q, k:      [batch, tokens, heads, dim] (k None: queries alone; its heads may
               be fewer) of one type, float32, float16 or bfloat16; any strides,
               such as views of one projection's output.
    positions: [tokens, axes] or [batch, tokens, axes], float32, int32 or int64;
               fractions and far positions keep their angle, which is reduced in
               fp64 and off by at most 2^-50 of the position.
    axes:      for each of 1 to 4 axes the number of elements of a head that turn
               by it, one part after the other: even, together at most dim (which
               is at most 512).  The elements behind them pass as they are.
    pairs:     pair i of a part of s elements, which turns by
               position * base^(-2 i / s): "adjacent" elements 2i and 2i + 1, or
               "halves" elements i and i + s / 2.

    Returns (q, k), new and contiguous.  Gradients of q and k are available,
    gradients of gradients and of positions are not."""
    kind = PAIRS.get(pairs)
    if kind is None:
        raise ValueError(f"pairs must be 'adjacent' or 'halves', got {pairs!r}")
    return _native().rotary(q, k, positions, axes, base, kind)


def attention(q, k, v, scale=None, causal=False, query_lengths=None, key_lengths=None):
    """Softmax attention, softmax(scale q k^T) v, without the matrix of scores
    ever in memory.

    q:     [batch, queries, heads, dim]; k, v: [batch, keys, kv_heads, dim], of one
           type, float32, float16 or bfloat16.  kv_heads divides heads: query head
           h uses key head h // (heads / kv_heads).  dim is a multiple of 8 to 128.
           Any strides: rows that do not lie at multiples of 16 bytes without gaps
           are copied first.
    scale: > 0; default dim ** -0.5.
    query_lengths, key_lengths: int32 [batch] on the same device: sequence b has
           that many queries and keys (clamped to 0 .. the tensor's); those behind
           them are not read.  Default: all.
    causal: query i sees key j <= i + (keys - queries) of its sequence: the last
           query sees the last key.

    Returns [batch, queries, heads, dim].  A query that sees no key, or is behind
    its sequence, gives zeros and takes a zero gradient.  Within the sequences' lengths
    queries, keys, values and the gradient that arrives must be finite: what is not
    may reach rows that do not see it.  Behind the lengths they may be anything.
    A query whose largest scaled score is above 10^9 (float16: 10^8) gives NaN, and one
    whose all are as far below 0 zeros: float32 does not tell them apart.
    Scores and sums are float32 (a probability that the backward forms again is off by some
    2^-23 of its score); for half types the probabilities (and in the
    backward, which forms them again, their gradients) are rounded to the type.
    Gradients of q, k and v are available, the same bits every time; gradients of
    gradients are not."""
    return _native().attention(q, k, v, scale, bool(causal), query_lengths, key_lengths)


def gated_linear(x, w_gate, w_up, b_gate=None, b_up=None, act="silu"):
    """The gated layer of a feed-forward block, both projections, the activation
    and the product in one kernel:

        act(x w_gate^T + b_gate) * (x w_up^T + b_up)

    x: [..., width]; w_gate, w_up: [hidden, width]; b_gate, b_up: [hidden] or None;
    contiguous, of one type, float32, float16 or bfloat16.
    act: "silu", "gelu" (with the error function) or "sigmoid".

    Returns [..., hidden].  Sums are float32, and where gradients are wanted the two
    projections are kept in float32 for the backward, whose gradients of them are
    rounded to the type before the products (float16: times a power of two that brings the
    largest into its range).  Gradients of all inputs are
    available, gradients of gradients are not."""
    kind = GATED_ACT.get(act)
    if kind is None:
        raise ValueError(f"act must be 'silu', 'gelu' or 'sigmoid', got {act!r}")
    return _native().gated_linear(x, w_gate, w_up, b_gate, b_up, kind)
