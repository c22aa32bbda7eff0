"""Plain fp64 definitions of rows held as e4m3 and of the product's epilogue.
Test infrastructure only, numpy alone.

A row v is held as e4m3 numbers y and one fp32 scale t / 448 with
t = max(max |v|, 448 * 2^-126) and y = e4m3(448 v / t).  The epilogue is
act(z + bias) + residual; SwiGLU's columns come in blocks of 16 gates and then
the 16 up values of the same features.
"""
from __future__ import annotations

import math

import numpy as np

from .longctx import E4M3, e4m3_codes

LEAST_TOP = 448.0 * 2.0 ** -126
_erfc = np.vectorize(math.erfc, otypes=[np.float64])


def quantise(v):
    """(codes uint8, scale float32) of rows of v (float64, along the last axis)."""
    v = np.asarray(v, np.float64)
    fine = np.isfinite(v).all(-1)
    v = np.where(fine[..., None], v, 0.0)
    t = np.maximum(np.abs(v).max(-1), LEAST_TOP)
    codes = e4m3_codes(448.0 * v / t[..., None])
    codes = np.where(fine[..., None], codes, 0).astype(np.uint8)
    return codes, np.where(fine, t / 448.0, np.nan).astype(np.float32)


def numbers(codes):
    """The e4m3 numbers of codes other than 0x7f and 0xff."""
    codes = np.asarray(codes)
    return np.where(codes & 0x80, -1.0, 1.0) * E4M3[codes & 0x7f]


def sigmoid(z):
    e = np.exp(-np.abs(z))
    return np.where(z >= 0, 1.0, e) / (1.0 + e)


def activation(z, act):
    if act == "relu":
        return np.maximum(z, 0.0)
    if act == "gelu":
        return 0.5 * z * _erfc(-z / math.sqrt(2.0))
    if act == "gelu_tanh":
        return z * sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3))
    if act == "silu":
        return z * sigmoid(z)
    return z


def gate_up(z):
    """(gates, ups), [M, N/2] each, of columns in blocks of 16 and 16."""
    b = z.reshape(z.shape[0], -1, 2, 16)
    return b[:, :, 0].reshape(z.shape[0], -1), b[:, :, 1].reshape(z.shape[0], -1)


def product(a, w, bias=None, residual=None, act="none"):
    """act(a w^T + bias) + residual; a [M, K], w [N, K] as float64 values."""
    z = a @ w.T
    if bias is not None:
        z = z + bias
    if act == "swiglu":
        g, u = gate_up(z)
        z = activation(g, "silu") * u
    else:
        z = activation(z, act)
    return z if residual is None else z + residual


def product_bound(a, w, bias=None, residual=None, act="none"):
    """How far a kernel may be from product(): a, w the operands' values.

    - The sum: at most K additions, each losing at most one unit in the last
      place (2^-23) of a partial sum of magnitudes; three more operations
      (two scales, bias) of half a unit each.
    - act has a slope of at most 1.13 (GELU's largest is 1.129, SiLU's 1.100).
    - Its evaluation: erfc, exp and a quotient of a few units each, and an
      argument off by 2 units, which moves erfc(x) by 2 x^2 and exp(x) by x
      units: below 2^-14 relative for |x| <= 88 and erfc's x <= 9.3, past
      which the result is below 2^-120.  A factor below 2^-126 counts as zero,
      at most 88 * 2^-126 < 2^-119 of a result (times |u| with SwiGLU).
    - The residual's addition, half a unit; then one rounding to bf16 (2^-8).
    """
    K = a.shape[1]
    mag = np.abs(a) @ np.abs(w).T
    z = a @ w.T
    b = 0.0 if bias is None else bias
    ez = (K + 3) * 2.0 ** -23 * (mag + np.abs(b))
    z = z + b
    if act == "swiglu":
        (g, u), (eg, eu) = gate_up(z), gate_up(ez)
        s = activation(g, "silu")
        r = s * u
        e = 1.13 * eg * (np.abs(u) + eu) + np.abs(s) * eu + 2.0 ** -14 * np.abs(r) \
            + 2.0 ** -119 * np.abs(u)
    else:
        r = activation(z, act)
        e = 1.13 * ez + (2.0 ** -14 * np.abs(r) if act not in ("none", "relu") else 0.0)
    if residual is not None:
        r = r + residual
        e = e + 2.0 ** -23 * np.abs(r)
    return e + 2.0 ** -8 * (np.abs(r) + e) + 2.0 ** -118
