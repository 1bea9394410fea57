"""64-bit definition of the INT8 feed-forward operators (numpy), and bounds on
what a correct kernel may differ from it by.

Codes and scales follow the fp32 rule exactly (whole numbers and fp32 values);
the sums of codes are whole numbers below 2^31, exact in 64 bits.  What rounds
in a kernel, and is bounded here:

  g, u       two fp32 products and one conversion of the sum: each at most 2^-24
             relative, together 3 x 2^-24
  act(g)     the exponential and the reciprocal are good to a few units: 2^-20
             relative is allowed for, and the change of act from g's own error
  y, h       one rounding to the 16-bit type on top
  combine    per slot 3 products and one fused addition in fp32, topk <= 16

A hidden value that lies next to the border of two 16-bit values may round to
either, and its code may then differ by one; ``down`` finds those and bounds
what they change.
"""
import math

import numpy as np

EPS16 = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11}  # half a step of the 16-bit type, relative
TINY16 = {"bf16": 2.0 ** -134, "fp16": 2.0 ** -25}  # half a step below its normal range


def quantise(x):
    """x: 16-bit values as float64 [M, K].  Returns (codes as float64, scales as float64)."""
    x = np.asarray(x, dtype=np.float64)
    bad = ~np.isfinite(x).all(axis=1)
    amax = np.abs(np.where(np.isfinite(x), x, 0.0)).max(axis=1)
    s = (amax.astype(np.float32) / np.float32(127)).astype(np.float32)
    with np.errstate(divide="ignore", invalid="ignore", over="ignore"):
        q = np.rint((x.astype(np.float32) / s[:, None]).astype(np.float32))
    q = np.where((amax == 0)[:, None] | bad[:, None], 0.0, np.clip(q.astype(np.float64), -127, 127))
    s = np.where(bad, np.nan, s.astype(np.float64))
    return q, s


def _sigmoid(v):
    e = np.exp(-np.abs(v))
    return np.where(v >= 0, 1.0 / (1.0 + e), e / (1.0 + e))


def act(g, kind):
    """(act(g), |act'(g)|), kind 0: silu, 1: gelu in its tanh form."""
    if kind == 0:
        p, q = _sigmoid(g), _sigmoid(-g)
        return g * p, np.abs(p + g * p * q)
    c = math.sqrt(8.0 / math.pi)
    v = c * (g + 0.044715 * g ** 3)
    p, q = _sigmoid(v), _sigmoid(-v)
    return g * p, np.abs(p + g * p * q * c * (1.0 + 0.134145 * g ** 2))


def front(q, s, w13, s13, kind, dt):
    """act(g) u in 64 bits, the bound on a kernel's fp32 value and that on its 16-bit value."""
    I = w13.shape[0] // 2
    acc = q @ np.asarray(w13, dtype=np.float64).T
    gu = acc * s[:, None] * np.asarray(s13, dtype=np.float64)
    g, u = gu[:, :I], gu[:, I:]
    a, da = act(g, kind)
    y = a * u
    e = 3 * 2.0 ** -24
    # the logistic's argument v carries at most 4 roundings, |g v'| <= 4 |g|^3 + |g| where p q is not negligible
    fp32 = np.abs(u) * (da * np.abs(g) * e + np.abs(a) * (2.0 ** -20 + e)) + np.abs(y) * 2.0 ** -23
    v = np.abs(g) if kind == 0 else 1.6 * np.abs(g) * (1 + 0.045 * g ** 2)
    fp32 += np.abs(y) * np.minimum(v, 90.0) * 4 * 2.0 ** -23  # act's relative change with an error in v
    # the logistic is taken from an exponential in (0, 1] whose result the hardware gives as 0 below 2^-126, the smallest
    # normal value: the logistic is off by less than that, act by |g| times it, y by |g u| times it
    fp32 += np.abs(g * u) * 2.0 ** -126
    return y, fp32, fp32 + np.abs(y) * EPS16[dt] * (1 + 2.0 ** -8) + TINY16[dt] + 2.0 ** -126


def route(logits, topk, mode):
    """ids and weights of the topk largest logits, equal ones to the lower expert; NaN and -inf mask."""
    logits = np.asarray(logits, dtype=np.float64)
    M, E = logits.shape
    ids = np.full((M, topk), -1, dtype=np.int32)
    gw = np.zeros((M, topk))
    for t in range(M):
        live = [e for e in range(E) if logits[t, e] > -np.inf]
        order = sorted(live, key=lambda e: (-logits[t, e], e))
        if not order:
            continue
        top = logits[t, order[0]]

        def ex(e):
            return 1.0 if logits[t, e] == top else math.exp(logits[t, e] - top)

        pick = order[:topk]
        total = sum(ex(e) for e in (pick if mode == 0 else order))
        for j, e in enumerate(pick):
            ids[t, j] = e
            gw[t, j] = ex(e) / total
    return ids, gw


def round16(v, dt):
    """float64 -> the 16-bit type (one rounding, ties to even), as float64."""
    v = np.asarray(v, dtype=np.float64)
    if dt == "fp16":
        with np.errstate(over="ignore"):
            return v.astype(np.float16).astype(np.float64)
    from .compare import f64_to_bf16_val
    return f64_to_bf16_val(v)


def _dequantised(h):
    """Codes times scale of each row, and the scales."""
    q, s = quantise(h)
    return q * s[:, None], s


def down(h, err, w2, s2, dt):
    """One expert: its 16-bit hidden rows known to lie within err of h before they are rounded.  Returns their down
    projection in 64 bits, the sum of the magnitudes, and what a hidden value that rounds, or is quantised, to the
    other neighbour can change."""
    w, s2 = np.asarray(w2, dtype=np.float64), np.asarray(s2, dtype=np.float64)
    near = [round16(h, dt), round16(h - err, dt), round16(h + err, dt)]
    ref, s = _dequantised(near[0])
    tol = np.zeros_like(ref)
    amax = [np.abs(v).max(axis=1) for v in near]
    for v in near:
        for a in amax:  # the row's maximum may be the neighbour too; its own code is 127 either way
            sa = (a.astype(np.float32) / np.float32(127)).astype(np.float64)
            with np.errstate(divide="ignore", invalid="ignore"):
                q = np.where(sa[:, None] > 0, np.clip(np.rint((v / sa[:, None]).astype(np.float32)), -127, 127), 0.0)
            tol = np.maximum(tol, np.abs(q * sa[:, None] - ref))
    tol[tol < np.abs(ref) * 2.0 ** -30] = 0.0
    return (ref @ w.T) * s2, (np.abs(ref) @ np.abs(w).T) * np.abs(s2), (tol @ np.abs(w).T) * np.abs(s2)


def layer(x, ids, gw, w13, s13, w2, s2, kind, dt):
    """The routed layer from ids and gw: (y in 64 bits, bound on a kernel's 16-bit y)."""
    M, topk = ids.shape
    E, H = s2.shape
    q, s = quantise(x)
    y, tol = np.zeros((M, H)), np.zeros((M, H))
    for e in range(E):
        t, j = np.nonzero(ids == e)
        if not len(t):
            continue
        h, err, _ = front(q[t], s[t], w13[e], s13[e], kind, dt)
        part, size, flips = down(h, err, w2[e], s2[e], dt)
        g = np.asarray(gw, dtype=np.float64)[t, j][:, None]
        for r, k in enumerate(t):
            y[k] += g[r] * part[r]
            # conversion, two products and the fused addition, and the additions of the slots
            tol[k] += np.abs(g[r]) * (flips[r] + size[r] * (4 + topk) * 2.0 ** -24)
    return y, tol + (np.abs(y) + tol) * EPS16[dt] + TINY16[dt] + 2.0 ** -126
