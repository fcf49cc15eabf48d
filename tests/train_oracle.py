"""The training operators in 64 bits on the CPU, from their definitions, and
how far a result in 32 bits may be off.

U = 2^-24 is half a step of fp32 relative to the value.  The bounds count
roundings (each at most U relative to its result) and carry them through the
formulas to first order, so they hold for every input without being fitted to
a result.  A result of a narrower type adds half a step of that type.
"""
from __future__ import annotations

import torch

U = 2.0 ** -24
TINY = {torch.float32: 2.0 ** -149, torch.float16: 2.0 ** -24, torch.bfloat16: 2.0 ** -133}


def rounding(value, dtype):
    """Half a step of `dtype` at `value`, subnormal steps included."""
    return value.abs() * (torch.finfo(dtype).eps / 2) + TINY[dtype] / 2


def check(got, want, bound, what):
    got = got.detach().cpu().double()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    off = (got - want).abs()
    bad = ~(off <= bound)
    if bad.any():
        at = int(torch.argmax(torch.where(bad, off / bound.clamp_min(1e-300), 0.0)))
        raise AssertionError(
            f"{what}: {int(bad.sum())} of {bad.numel()} values are off; at {at}: "
            f"{got.flatten()[at]:.9e} for {want.flatten()[at]:.9e}, "
            f"off {off.flatten()[at]:.3e}, bound {bound.expand_as(off).flatten()[at]:.3e}")


# ------------------------------------------------------------------ clipping and AdamW
def norm_of(grads):
    return torch.stack([g.double().square().sum() for g in grads]).sum().sqrt()


def factor(norm, max_norm):
    return torch.clamp(max_norm / (norm + 1e-6), max=1.0)


def check_norm(got, want):
    check(got, want, want * U * 1.01 + TINY[torch.float32], "norm")


def clipped(g, c):
    """c g and its bound: the factor rounded to fp32, the product, the type."""
    want = g.double() * c
    bound = want.abs() * 2 * U * 1.01 + rounding(want, g.dtype)
    return want, bound


def adamw(p, w, m, v, g, c, lr, beta1, beta2, eps, decay, t):
    """New (p, w, m, v), each with its bound.  w: the fp32 weights, or None
    (then p's own values)."""
    base = (p if w is None else w).double()
    g = g.double() * c  # 2 roundings: the factor, the product
    a, b = beta1 * m.double(), (1 - beta1) * g
    m1 = a + b
    # a: beta1.  b: g' 2, the factor, the product.  the sum
    tol_m = (a.abs() + b.abs()) * 6 * U + TINY[torch.float32]
    v1 = beta2 * v.double() + (1 - beta2) * g * g
    # g'^2 4, the factor, two products, beta2, the sum
    tol_v = v1 * 10 * U + 4 * TINY[torch.float32]
    root = (v1 / (1 - beta2 ** t)).sqrt()
    # a square below the smallest fp32 vanishes
    tol_root = root * 8 * U + (8 * TINY[torch.float32] / (1 - beta2 ** t)) ** 0.5
    denom = root + eps
    size = lr / (1 - beta1 ** t)
    step = size * m1 / denom
    w1 = base * (1 - lr * decay) - step
    mag = size * (a.abs() + b.abs()) / denom
    # the step: m 6, the root (above), eps, the sum, the quotient, size, the product.  w: the decay, its product, the sum
    tol_w = mag * 12 * U + size * m1.abs() / denom ** 2 * tol_root + 3 * U * (base.abs() + mag) \
        + 4 * TINY[torch.float32]
    tol_p = tol_w + (rounding(w1, p.dtype) * 1.01 if p.dtype != torch.float32 else 0.0)
    return (w1, tol_p), (w1, tol_w), (m1, tol_m), (v1, tol_v)


# ------------------------------------------------------------------ the joint between two blocks
def activate(g, act):
    return torch.sigmoid(g) if act == "sigmoid" else g


def joint(x, branch, gate, scale, post, pre, eps, act):
    """(residual, normed) of 64-bit inputs; None: 1."""
    bh = branch / torch.sqrt(branch.square().mean(-1, keepdim=True) + eps)
    for w in (scale, post):
        bh = bh if w is None else bh * w
    r = x + (bh if gate is None else bh * activate(gate, act))
    h = r / torch.sqrt(r.square().mean(-1, keepdim=True) + eps)
    return r, h if pre is None else h * pre


class Joint:
    """The joint of given inputs with all gradients and their bounds."""

    # A row's sum of positive terms: a thread adds at most 32 of its own one
    # after another, then 6 steps over the wave and 8 over the workgroup.
    CHAIN = 46

    def __init__(self, x, branch, gate, scale, post, pre, eps, act, dr, dh):
        types = (x.dtype, branch.dtype)
        one = torch.ones((), dtype=torch.float64)

        def d(t):
            return one if t is None else t.detach().cpu().double()

        x, b, c, w = d(x), d(branch), d(scale) * d(post), d(pre)
        half = types[1] != torch.float32
        gd = None if gate is None else d(gate)
        a = one if gate is None else activate(gd, act)
        # act: the exponential, the sum, the quotient; a fast exponential is off by its argument's rounding
        act_u = 0.0
        if gate is not None and act == "sigmoid":
            act_u = 6.0 + (2.0 * float(gd.abs().max()) if half else 0.0)

        def mean(t):
            return t.mean(-1, keepdim=True)

        ib = 1 / torch.sqrt(mean(b * b) + eps)
        bh = b * ib
        add = a * c * bh
        r = x + add
        ir = 1 / torch.sqrt(mean(r * r) + eps)
        rh = r * ir
        # a reciprocal root: half of (the sum, the mean, eps) and the root and the quotient
        root = (self.CHAIN + 2) / 2 + 3
        # r: the root, its product, c, a, two products, the sum
        tol_r = U * r.abs() + U * (root + 5 + act_u) * add.abs()
        share = torch.sqrt(mean(add * add) / mean(r * r).clamp_min(1e-300)).clamp(max=1e12)
        tol_ir = U * (root + 2 + (root + 5 + act_u) * share)  # relative
        h = rh * w
        tol_h = (tol_ir + 3 * U) * h.abs() + tol_r * ir * w.abs()
        self.residual = (r, tol_r + rounding(r, types[0]) * 1.01)
        self.normed = (h, tol_h + rounding(h, types[1]) * 1.01)

        dr, dh = (torch.zeros_like(r) if t is None else d(t) for t in (dr, dh))
        wd = dh * w
        m1 = mean(wd * rh)
        e = dr + ir * (wd - rh * m1)
        t = e * a * c
        db = ib * (t - bh * mean(t * bh))
        # what one factor of these may be off by, relative to the magnitudes (r's own share included)
        q = tol_ir + U * (root + 8 + act_u) + U * (root + 6 + act_u) * (add.abs() / r.abs().clamp_min(1e-300)).clamp(max=1.0)
        rmag = (r.abs() + add.abs()) * ir  # |rh| where x and the branch cancel
        k_e = 4 * q + (self.CHAIN + 10) * U
        e_mag = dr.abs() + ir * wd.abs() + rmag * ir * mean(wd.abs() * rmag)
        u_mag = dr.abs() + ir * wd.abs()
        add_mag = add.abs()
        m2_mag = mean(u_mag * add_mag) + ir * mean(wd.abs() * rmag) * mean(rmag * add_mag)
        k_b = k_e.amax(-1, keepdim=True) * 2
        ac = (a * c).abs()
        self.grads = {
            "x": (e, k_e * e_mag + rounding(e, types[0]) * 1.01),
            "branch": (db, k_b * ib * (e_mag * ac + bh.abs() * m2_mag) + rounding(db, types[1]) * 1.01)}
        rows = tuple(range(r.dim() - 1))
        count = r[..., 0].numel()

        def over_rows(t):
            return t.expand_as(r).reshape(count, -1).sum(0)

        total, total_mag = over_rows(e * a * bh), over_rows(k_b * e_mag * (a * bh).abs())
        chain = U * (count + 8) * over_rows(e_mag * (a * bh).abs())
        s, p_ = (torch.ones_like(total) if t is None else d(t) for t in (scale, post))
        self.grads["scale"] = (total * p_, (total_mag + chain) * p_.abs() + rounding(total * p_, torch.float32))
        self.grads["post_weight"] = (total * s, (total_mag + chain) * s.abs() + rounding(total * s, torch.float32))
        dpre = over_rows(dh * rh)
        self.grads["pre_weight"] = (dpre, over_rows((k_e + U * (count + 8)) * dh.abs() * rmag)
                                    + rounding(dpre, torch.float32))
        if gate is not None:
            slope = a * (1 - a) if act == "sigmoid" else torch.ones_like(a)
            slope_mag = a if act == "sigmoid" else slope
            dg = e * c * bh * slope
            bound = (k_b + U * (count + 8)) * e_mag * (c * bh).abs() * slope_mag
            shared = tuple(k for k in rows if gd.shape[k] != r.shape[k])
            if shared:
                dg, bound = dg.sum(shared, keepdim=True), bound.sum(shared, keepdim=True)
            self.grads["gate"] = (dg, bound + rounding(dg, types[1]) * 1.01)
