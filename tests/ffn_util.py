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
