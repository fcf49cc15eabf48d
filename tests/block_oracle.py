"""Rotary positions, attention and the gated layer in 64 bits on the CPU, from
their definitions, and how far a result may be off.

U = 2^-24 is half a step of fp32.  The bounds count roundings to first order and
carry them through the formulas by magnitudes, so they hold for every input.  A
sum of n products is counted with 2 U for each term (a matrix instruction may cut
where an addition rounds).  Where a half type is rounded to on the way (the
probabilities, the gradients of scores and projections), half a step of that type
is counted; a result adds half a step of its own.
"""
from __future__ import annotations

import math

import torch

from train_oracle import TINY, U, check, rounding  # noqa: F401

SLACK = 1.02  # what first order leaves out
# The exponential instruction gives 0 where the result is below fp32's smallest normal
# number, and a matrix instruction may take such an operand or sum for 0: a probability, a
# gradient of a score and a result are each off by at most this.
LEAST = 2.0 ** -126


def half_step(dtype):
    """Of a half type, relative; 0 for fp32, whose roundings are counted one by one."""
    return 0.0 if dtype == torch.float32 else torch.finfo(dtype).eps / 2


def d(t):
    return None if t is None else t.detach().cpu().double()


# ------------------------------------------------------------------ rotary positions
def pairs_of(axes, kind):
    first, second, rate, axis, at = [], [], [], [], 0
    for a, size in enumerate(axes):
        for i in range(size // 2):
            first.append(at + (2 * i if kind == "adjacent" else i))
            second.append(at + (2 * i + 1 if kind == "adjacent" else i + size // 2))
            rate.append(-2.0 * i / size)
            axis.append(a)
        at += size
    return first, second, torch.tensor(rate, dtype=torch.float64), axis


def rotary(x, positions, axes, base, kind, way=1.0):
    """(the turned x, its bound)."""
    first, second, rate, axis = pairs_of(axes, kind)
    v, p = d(x), positions.detach().cpu().double()
    angle = way * (p[..., axis] * torch.exp(rate * math.log(base))).unsqueeze(-2)
    c, s = angle.cos(), angle.sin()
    out, mag = v.clone(), torch.zeros_like(v)
    out[..., first] = v[..., first] * c - v[..., second] * s
    out[..., second] = v[..., second] * c + v[..., first] * s
    both = v[..., first].abs() + v[..., second].abs()
    mag[..., first] = both
    mag[..., second] = both
    # a sine: the rate's and the angle's roundings in 64 bits, the reduced angle's to fp32, the function's 4 U; two products, the sum
    far = float(p.abs().max()) if p.numel() else 0.0
    bound = mag * (8 * U + far * 2.0 ** -50) + torch.where(mag > 0, rounding(out, x.dtype) * SLACK, 0.0)
    return out, bound


# ------------------------------------------------------------------ attention
def seen_by(n, m, causal, ql, kl):
    """[n, m]: query i sees key j."""
    i, j = torch.arange(n)[:, None], torch.arange(m)[None]
    seen = (i < ql) & (j < kl)
    return seen & (j <= i + (kl - ql)) if causal else seen


class Attention:
    """out and, with d_out, the gradients, each with its bound."""

    def __init__(self, q, k, v, scale=None, causal=False, query_lengths=None, key_lengths=None, d_out=None):
        dtype, t = q.dtype, half_step(q.dtype)
        tiny = TINY[dtype] / 2 if dtype == torch.float16 else 0.0
        (batch, n, heads, dim), m, kv = q.shape, k.shape[1], k.shape[2]
        scale = dim ** -0.5 if scale is None else scale
        qd, kd, vd, dod = d(q), d(k), d(v), d(d_out)
        names = ("out", "q", "k", "v")
        value = dict(zip(names, (torch.zeros_like(x) for x in (qd, qd, kd, vd))))
        off = {key: torch.zeros_like(x) for key, x in value.items()}
        clamp = lambda lengths, b, most: most if lengths is None else min(max(int(lengths[b]), 0), most)
        for b in range(batch):
            ql, kl = clamp(query_lengths, b, n), clamp(key_lengths, b, m)
            seen = seen_by(n, m, causal, ql, kl)
            live = seen.any(1, keepdim=True)
            for h in range(heads):
                c = h // (heads // kv)
                # (what is behind a sequence is not read)
                Q, K, V = qd[b, :, h].clone(), kd[b, :, c].clone(), vd[b, :, c].clone()
                Q[ql:], K[kl:], V[kl:] = 0, 0, 0
                s = scale * (Q @ K.t())
                s_mag = scale * (Q.abs() @ K.abs().t())
                s = torch.where(seen, s, -math.inf)
                lse = torch.logsumexp(s, 1, keepdim=True)
                p = torch.where(live, torch.exp(s - torch.where(live, lse, 0.0)), 0.0)
                # a probability: its score and the row's sum, each through the worst of the row's scores; the
                # exponent's roundings (2 of each of the score and the statistic), the exponential; the sum's
                worst = torch.where(seen, s_mag, 0.0).amax(1, keepdim=True)
                size = torch.where(live, lse.abs(), 0.0) + worst
                rel = 2 * (2 * dim + 4) * U * worst + 8 * U * size + (2 * m + 20) * U
                rel = torch.where(live, rel, 0.0)
                o = p @ V
                o_off = (rel + t + 2 * m * U) * (p @ V.abs()) + (tiny + LEAST) * (seen.double() @ V.abs()) + 4 * U * o.abs() + LEAST
                value["out"][b, :, h] = o
                off["out"][b, :, h] = o_off + rounding(o, dtype) * SLACK
                if dod is None:
                    continue
                do = dod[b, :, h].clone()
                do[ql:] = 0
                # (2^-39: half a step of the smallest fp16 number, of a probability times 2^14)
                rel_p = rel + t
                dv = p.t() @ do
                dv_off = (p * (rel_p + 2 * n * heads * U)).t() @ do.abs() + (tiny * 2.0 ** -14 + LEAST) * (seen.double().t() @ do.abs()) + LEAST
                dp, dp_mag = do @ V.t(), do.abs() @ V.abs().t()
                delta, delta_mag = (do * o).sum(1, keepdim=True), (do * o).abs().sum(1, keepdim=True)
                # (delta takes the output with what its rounding left)
                o_err = (do.abs() * (o_off + (t * t if t else U) * o.abs() + TINY[dtype])).sum(1, keepdim=True)
                ds = p * (dp - delta)
                ds_off = p * ((dp.abs() + delta.abs()) * (rel_p + 4 * U) + 2 * dim * U * (dp_mag + delta_mag) + o_err)
                ds_off = ds_off + t * ds.abs() + torch.where(seen, tiny + LEAST * (1 + dp.abs() + delta.abs()), 0.0)
                value["q"][b, :, h] = scale * (ds @ K)
                off["q"][b, :, h] = scale * (ds_off @ K.abs() + 2 * (m + 2) * U * (ds.abs() @ K.abs()))
                value["k"][b, :, c] += scale * (ds.t() @ Q)
                off["k"][b, :, c] += scale * (ds_off.t() @ Q.abs() + 2 * (n * heads + 2) * U * (ds.abs().t() @ Q.abs()))
                value["v"][b, :, c] += dv
                off["v"][b, :, c] += dv_off
        for key in ("q", "k", "v"):
            off[key] = off[key] + rounding(value[key], dtype) * SLACK + LEAST
        self.value, self.off = value, {key: x * SLACK for key, x in off.items()}

    def check(self, which, got):
        check(got, self.value[which], self.off[which], which)


# ------------------------------------------------------------------ the gated layer
def act_of(g, act):
    """act(g), act'(g), and the largest |act'| and |act''| there are."""
    if act == "gelu":
        phi = 0.5 * torch.erfc(-g / math.sqrt(2))
        pdf = torch.exp(-0.5 * g * g) / math.sqrt(2 * math.pi)
        return g * phi, phi + g * pdf, 1.13, 0.8
    a, b = torch.sigmoid(g), torch.sigmoid(-g)
    return (a, a * b, 0.25, 0.1) if act == "sigmoid" else (g * a, a * (1 + g * b), 1.1, 0.5)


class Gated:
    """out and, with d_out, the gradients, each with its bound."""

    def __init__(self, x, w_gate, w_up, b_gate=None, b_up=None, act="silu", d_out=None):
        dtype, t = x.dtype, half_step(x.dtype)
        X, G, W = d(x).reshape(-1, x.shape[-1]), d(w_gate), d(w_up)
        rows, width = X.shape
        hidden = G.shape[0]

        def projected(w, b):
            y, mag = X @ w.t(), X.abs() @ w.abs().t()
            off = 2 * (width + 2) * U * mag
            if b is None:
                return y, off
            return y + d(b), off + 2 * U * (y.abs() + d(b).abs())

        (g, g_off), (u, u_off) = projected(G, b_gate), projected(W, b_up)
        a, slope, top, bend = act_of(g, act)
        # the activation: a fast exponential is off by its argument's rounding, the quotient and products
        a_rel = (12 + 3 * g.abs().clamp(max=100.0)) * U
        if act == "gelu" and t > 0:
            # a half type's error function: 8 U of itself (a fit's error and its evaluation), and its
            # exponential's argument g^2 / 2 log2 e < 0.73 g^2 rounded twice
            a_rel = a_rel + (8 + 1.5 * (g * g).clamp(max=400.0)) * U
        a_off = top * g_off + a_rel * a.abs()
        h = a * u
        h_off = a_off * u.abs() + a.abs() * u_off + 2 * U * h.abs()
        shape = (*x.shape[:-1], hidden)
        self.value = {"out": h.reshape(shape)}
        self.off = {"out": (h_off + rounding(h, dtype) * SLACK).reshape(shape)}
        if d_out is not None:
            dh = d(d_out).reshape(-1, hidden)
            slope_off = bend * g_off + (16 + 3 * g.abs().clamp(max=100.0)) * U * (slope.abs() + g.abs().clamp(max=1.0))
            dg, du = dh * u * slope, dh * a
            dg_off = dh.abs() * (u.abs() * slope_off + u_off * slope.abs()) + 3 * U * dg.abs()
            du_off = dh.abs() * a_off + 2 * U * du.abs()
            if b_gate is not None or b_up is not None:
                for name, value, off in (("b_gate", dg, dg_off), ("b_up", du, du_off)):
                    s = value.sum(0)
                    self.value[name] = s
                    self.off[name] = off.sum(0) + (rows + 4) * U * value.abs().sum(0) + rounding(s, dtype) * SLACK
            dg_off, du_off = dg_off + rounding(dg, dtype) * (t > 0), du_off + rounding(du, dtype) * (t > 0)
            dx = dg @ G + du @ W
            dx_off = dg_off @ G.abs() + du_off @ W.abs() + 2 * (2 * hidden + 2) * U * (dg.abs() @ G.abs() + du.abs() @ W.abs())
            self.value["x"] = dx.reshape(x.shape)
            self.off["x"] = (dx_off + rounding(dx, dtype) * SLACK).reshape(x.shape)
            for name, value, off in (("w_gate", dg, dg_off), ("w_up", du, du_off)):
                dw = value.t() @ X
                self.value[name] = dw
                self.off[name] = off.t() @ X.abs() + 2 * (rows + 2) * U * (value.abs().t() @ X.abs()) + rounding(dw, dtype) * SLACK
        self.off = {key: v * SLACK for key, v in self.off.items()}

    def check(self, which, got):
        check(got, self.value[which], self.off[which], which)
