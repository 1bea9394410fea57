"""Plain 64-bit forms of the 4-bit weight operators (numpy, no product code).

W[n, k] = ws[n, k // G] * (code[n, k] - zero[n, k // G]); codes two a byte, element
2i in the low nibble; zero 8 where there are no zero points.  Every function takes
float64 arrays that hold the 16-bit inputs' values exactly and returns the exact
result with what a tolerance needs:

  S  sum |ws| (code + zero) |x| over the reduction (rounding of the running fp32 sums),
  Q  sqrt(sum (w x)^2)            (independent roundings of the weights).
"""
from __future__ import annotations

import numpy as np

HALF_STEP = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11}  # largest relative rounding error of the type


def dense(w, ws, wz, group):
    """float64 [N, K] from codes uint8 [N, K/2], ws [N, K/G], wz [N, K/G] or None."""
    codes = np.stack([w & 15, w >> 4], axis=2).reshape(len(w), -1).astype(np.float64)
    zero = 8.0 if wz is None else np.repeat(wz.astype(np.float64), group, axis=1)
    return np.repeat(ws, group, axis=1) * (codes - zero)


def dense_parts(w, ws, wz, group):
    """|ws| (code + zero): what the sums add up where the zero is taken out after the sum."""
    ones = np.abs(ws)
    zero = 8.0 if wz is None else wz.astype(np.float64)
    return np.abs(dense(w, ones, np.zeros(ws.shape, np.uint8), group)) + np.repeat(ones * zero, group, axis=1)


def product(x, W, parts):
    """x [M, R] times W [R, C]: (exact, S, Q); parts as dense_parts, shaped like W."""
    return x @ W, np.abs(x) @ parts, np.sqrt((x * x) @ (W * W))


def sum_tolerance(S, Q, R, dtype, weights_exact):
    """Bound on a kernel's fp32 sum against the exact one.

    fp32: R + 8 additions and products, each within 2^-24 of partial sums that are
    at most S in absolute value (sums of code * x and of zero * x, times the scale).
    Weights rounded to the 16-bit type first: R independent errors of at most
    h |w x|; by Hoeffding's inequality the sum exceeds 7 h Q with probability
    2 exp(-24.5) = 5e-11.
    """
    h = 0.0 if weights_exact else HALF_STEP[dtype]
    return 7.0 * h * Q + (R + 8) * 2.0 ** -24 * S


def rounded_tolerance(y, E, dtype):
    """|r16(v) - y| for |v - y| <= E: half a step of the type, or of its smallest numbers."""
    tiny = 2.0 ** -25 if dtype == "fp16" else 2.0 ** -134
    return HALF_STEP[dtype] * (np.abs(y) + E) + E + tiny


def act(g, kind):
    """act(g) and act'(g); kind 0: silu, 1: gelu in its tanh form.

    Both are g times a logistic p = 1 / (1 + e^-v); 0.5 (1 + tanh z) is written as
    that logistic of 2 z, since 1 + tanh z has no digits left for z below -15."""
    c = np.sqrt(8.0 / np.pi)
    v, dv = (g, 1.0) if kind == 0 else (c * (g + 0.044715 * g ** 3), c * (1.0 + 3 * 0.044715 * g * g))
    p, q = 1.0 / (1.0 + np.exp(-v)), 1.0 / (1.0 + np.exp(v))
    return g * p, p + g * p * q * dv


# |act'| <= 1.13 and |act''| <= 1.2 for both activations (silu 1.0999 / 0.5, gelu 1.129 / 1.13)
ACT_D1, ACT_D2 = 1.13, 1.2
# v_exp_f32, v_rcp_f32 and a few products on the way to p, q: 16 fp32 ulps, relative to act and
# act', plus |v| 2^-23 relative for the exponent's argument
ACT_REL = 32 * 2.0 ** -24


def gate_tolerance(g, u, Eg, Eu, kind):
    """Bounds on act(g) u where g, u are off by Eg, Eu, and on the activation's own error."""
    a, da = act(g, kind)
    rel = ACT_REL + (np.abs(g) + 0.1 * np.minimum(np.abs(g), 30.0) ** 3) * 2.0 ** -23
    Ea = ACT_D1 * Eg + np.abs(a) * rel + 2.0 ** -126
    Eda = ACT_D2 * Eg + (np.abs(da) + np.abs(g) * 0.25) * rel
    return a, da, Ea, Eda
