"""The feed-forward operators' definitions in 64 bits, for the GPU tests."""

from __future__ import annotations

import math

import numpy as np

ACTS = {"none": 0, "relu": 1, "silu": 2, "gelu": 3, "gelu_tanh": 4}

# |act'| is at most 1 for relu, 1.0999 for silu, 1.1290 for both forms of gelu
LIPSCHITZ = 1.13


def act64(name, v):
    v = np.asarray(v, dtype=np.float64)
    with np.errstate(all="ignore"):
        if name == "relu":
            return np.where(v < 0, 0.0, v)
        if name == "silu":
            return v / (1.0 + np.exp(-v))
        if name == "gelu":
            return 0.5 * v * np.vectorize(math.erfc)(-v / math.sqrt(2.0))
        if name == "gelu_tanh":
            u = math.sqrt(2.0 / math.pi) * (v + 0.044715 * v ** 3)
            return v / (1.0 + np.exp(-2.0 * u))
    return v


def half_step(dt):
    """Relative half step of the output type (0: fp16, 1: bf16)."""
    return 2.0 ** -11 if dt == 0 else 2.0 ** -8


def epilogue64(f, act, bias=None, mul=None, res=None):
    v = f if bias is None else f + bias
    v = act64(act, v)
    v = v if mul is None else v * mul
    return v if res is None else v + res


def epilogue_bound(tol_f, f, act, dt, bias=None, mul=None, res=None):
    """Bound on |y - epilogue64(f)| where the fp32 f is off by at most tol_f per element:
    the activation stretches that by LIPSCHITZ, mul by its value; the fp32 steps after the
    product are each off by at most 2^-24 relative to their value, the activation by 8 such
    units (expf and erfcf are within 4, the quotient and products add theirs) plus, for
    v < 0, the 3 units of the exponent's argument u times |u'(v) v|, which is at most
    |v| (1.6 + 0.22 v^2) for the tanh form and less for the others; and the store by half
    a step of the type (fp16 values below 2^-14 are spaced 2^-24)."""
    b = 0.0 if bias is None else bias
    a = np.abs(act64(act, f + b))
    v = np.maximum(0.0, -(f + b))
    units = np.where(a > 0, 8 + 3 * v * (1.6 + 0.22 * v * v), 0.0)
    m = 1.0 if mul is None else np.abs(mul)
    r = 0.0 if res is None else np.abs(res)
    y = np.abs(epilogue64(f, act, bias, mul, res))
    fp32 = 2.0 ** -24 * (LIPSCHITZ * m * (np.abs(f) + np.abs(b)) + units * a * m + a * m + r)
    return LIPSCHITZ * tol_f * m + fp32 + half_step(dt) * (y + LIPSCHITZ * tol_f * m) + (2.0 ** -25 if dt == 0 else 0.0)


def product_bound(x, w, dt):
    """Bound on the error of x . w^T whose weights are rounded to the type and summed in fp32
    (x [m, K], w [n, K] in 64 bits).  The weights' roundings are independent, zero on average and at
    most half a step each, so their sum is within 7 u sqrt(sum x^2 w^2) except with probability
    2 exp(-49 / 2) = 5e-11 per element (Hoeffding); fp16 weights below 2^-14 are rounded to
    multiples of 2^-24.  The K additions and the decode's fp32 steps are each off by at most 2^-24 of
    what they add up to."""
    x2, w2, ax, aw = x * x, w * w, np.abs(x), np.abs(w)
    tol = 7 * half_step(dt) * np.sqrt(x2 @ w2.T) + (x.shape[1] + 4) * 2.0 ** -24 * (ax @ aw.T)
    if dt == 0:
        tol = tol + 7 * 2.0 ** -25 * np.sqrt(x2.sum(1, keepdims=True))
    return tol


def glu64(f, act, bias=None):
    f = f if bias is None else f + bias
    h = f.shape[1] // 2
    return act64(act, f[:, :h]) * f[:, h:]


def glu_bound(tol_f, f, act, dt, bias=None):
    """Bound on |y - glu64(f)|: the gate's error stretched by the activation times the up value,
    and the up value's error times the gate's."""
    h = f.shape[1] // 2
    b = np.zeros(f.shape[1]) if bias is None else bias
    gate, up = f[:, :h], f[:, h:] + b[h:]
    tg = epilogue_bound(tol_f[:, :h], gate, act, 1, b[:h]) - half_step(1) * (np.abs(act64(act, gate + b[:h])) + LIPSCHITZ * tol_f[:, :h])
    tu = tol_f[:, h:] + 2.0 ** -23 * (np.abs(f[:, h:]) + np.abs(b[h:]))
    a = np.abs(act64(act, gate + b[:h]))
    err = tg * (np.abs(up) + tu) + a * tu + 2.0 ** -23 * a * np.abs(up)
    return err + half_step(dt) * (a * np.abs(up) + err) + (2.0 ** -25 if dt == 0 else 0.0)
