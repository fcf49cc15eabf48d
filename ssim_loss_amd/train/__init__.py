"""The rest of a training step around the SSIM loss, on AMD MI355X: the global
gradient norm and clipping by it, AdamW with the clipping fused in, and the
joint between two blocks of an image network with its gradient.

The C ABI is ``include/ssim_train_amd.h``; ``_bind`` (csrc/bind.cpp) calls it on
torch tensors, on torch's current stream of their device.  The computation runs
in the HIP kernels of ``libssim_train_amd.so``; there is no fallback path.

  clip_grads_(grads, max_norm, out=None)  -> the gradients' global norm
  grad_norm(grads)                        -> the norm alone
  AdamW(params, ...).step(grads=None)     -> the norm before clipping, or None
  block_norm(x, branch, gate=..., ...)    -> (residual, normed), with autograd
"""
from __future__ import annotations

import ctypes
import os
import threading

from .. import SsimError
from ..build import BIND_PATH, TRAIN_LIB_PATH

# SSIM_TRAIN_ABI_VERSION of include/ssim_train_amd.h that this package follows
ABI_VERSION = 1

GATE_ACT = {"none": 0, "sigmoid": 1}

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
                    ("ssim_block_norm_backward", i32, [vp, vp, vp, vp, vp, vp, vp])):
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
