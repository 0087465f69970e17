"""Plain definitions in 64 bits of the feed-forward block's operators, for the
tests, written from the formulas in include/mm.h, with bounds on what 32-bit sums
and one rounding may add. torch tensors, on whatever device they lie.

U is half a step of f32. A sum of K products in f32, in any order, is off by at
most (K + 8) U sum|x w| (each product and each addition rounds once; 8 covers the
joining of partial sums). act has a slope of at most 1.13 and a second derivative
of at most 1.2 (both gates)."""
from __future__ import annotations

import math

import torch

NONE, SILU, GELU = 0, 1, 2
TORCH = {0: torch.float32, 1: torch.float16, 2: torch.bfloat16}
U = 2.0 ** -24
SLOPE, CURVE = 1.13, 1.2
C = 2 * math.sqrt(2 / math.pi)


def rounding(dtype: int, value):
    """Half a step of `value` in the type; a value below the smallest normal number has that number's step."""
    f = torch.finfo(TORCH[dtype])
    return f.eps / 2 * value.abs().clamp_min(f.tiny)


def _z(a, gate):
    """z(a) and its slope."""
    if gate == SILU:
        return a, torch.ones_like(a)
    return C * (a + 0.044715 * a ** 3), C * (1 + 3 * 0.044715 * a ** 2)


def act(a, gate):
    return a * torch.sigmoid(_z(a, gate)[0])


def act_slope(a, gate):
    z, dz = _z(a, gate)
    s, rest = torch.sigmoid(z), torch.sigmoid(-z)
    return s + a * s * rest * dz


def act_error(a, gate):
    """Of act(a) in f32: exp, one addition, one division and one product are 10 U of it; an error of 6 U |z| in the
    exponent's argument (its own rounding, and the cubic's) is as much of the sigmoid where that is small."""
    return (10 + 6 * _z(a, gate)[0].abs().clamp_max(110)) * U * act(a, gate).abs() + 1e-37


def products(x, w):
    """x w^T and the sum's error in f32."""
    x, w = x.double(), w.double()
    return x @ w.t(), (x.shape[1] + 8) * U * (x.abs() @ w.abs().t())


def gated(x, w, gate):
    """h, pre and the errors of both before rounding."""
    n = w.shape[0] // 2
    pre, e = products(x, w)
    g, u, eg, eu = pre[:, :n], pre[:, n:], e[:, :n], e[:, n:]
    h = act(g, gate) * u
    eh = SLOPE * eg * (u.abs() + eu) + act(g, gate).abs() * eu + act_error(g, gate) * u.abs() + 2 * U * h.abs()
    return h, pre, eh, e


def gated_grad(pre, e, dh, gate):
    """dpre and its error before rounding, from pre-activations with error e."""
    n, dh = pre.shape[1] // 2, dh.double()
    g, u, eg, eu = pre[:, :n], pre[:, n:], e[:, :n], e[:, n:]
    dg, du = dh * u * act_slope(g, gate), dh * act(g, gate)
    # the slope's own error: each term at most 0.6, ten roundings each, and 6 U |z| times a term that falls faster
    eg2 = dh.abs() * ((u.abs() + eu) * (CURVE * eg + 24 * U) + SLOPE * eu)
    eu2 = dh.abs() * (SLOPE * eg + act_error(g, gate)) + 2 * U * du.abs()
    return torch.cat((dg, du), 1), torch.cat((eg2 + 2 * U * dg.abs(), eu2), 1)


def quantise(x):
    """Codes and scales: the quotient of two 24-bit numbers in 64 bits has a tie only where it is one."""
    x = x.double()
    top = x.abs().amax(1)
    scale = (top / 127).to(torch.float32)
    scale = torch.where(scale < 2.0 ** -126, torch.full_like(scale, 2.0 ** -126), scale)
    return torch.round(x / scale.double()[:, None]).to(torch.int8), scale


def i8(q, s, w, ws, gate):
    """y and its error before rounding: three roundings of each scaled sum, the sum itself is exact."""
    y = (q.double() @ w.double().t()) * ws.double() * s.double()[:, None]
    if gate == NONE:
        return y, 3 * U * y.abs()
    n = w.shape[0] // 2
    g, u = y[:, :n], y[:, n:]
    h = act(g, gate) * u
    return h, 3 * U * SLOPE * g.abs() * u.abs() + act_error(g, gate) * u.abs() + 6 * U * h.abs()
