"""Gated activation, its backward pass and 8-bit checkpoints (oracle; test
infrastructure).

float64 throughout, but for what the library defines in binary32: a
checkpoint's scale and the quotients its codes round, and the value
``binary32(code * scale)`` that a code stands for.
"""

from __future__ import annotations

import math

import numpy as np

from . import formats as F
from .quantize import QMAX, div32

_erfc = np.vectorize(math.erfc, otypes=[np.float64])


def act(g: np.ndarray, kind: str):
    """act(g) and its derivative, float64."""
    g = np.asarray(g, np.float64)
    if kind == "silu":
        p = 1.0 / (1.0 + np.exp(-g))
        return g * p, p * (1.0 + g * (1.0 - p))
    cdf = 0.5 * _erfc(g / -math.sqrt(2.0))  # erfc, not 1 + erf: the lower tail does not cancel
    return g * cdf, cdf + g * np.exp(-0.5 * g * g) / math.sqrt(2.0 * math.pi)


def gated(gate_up: np.ndarray, kind: str) -> np.ndarray:
    """h = act(gate) * up of [M, 2 I]."""
    I = gate_up.shape[1] // 2
    return act(gate_up[:, :I], kind)[0] * np.asarray(gate_up[:, I:], np.float64)


def gated_backward(dh: np.ndarray, gate_up: np.ndarray, kind: str):
    """(d_gate_up, h) from the values of gate and up."""
    I = gate_up.shape[1] // 2
    up = np.asarray(gate_up[:, I:], np.float64)
    f, df = act(gate_up[:, :I], kind)
    dh = np.asarray(dh, np.float64)
    return np.concatenate([dh * up * df, dh * f], axis=1), f * up


def ue8m0_exponent(absmax: np.ndarray, code: str) -> np.ndarray:
    """Smallest e in [-127, 127] with absmax <= qmax * 2**e; 0 for an all-zero block."""
    a = np.asarray(absmax, np.float64)
    m, e = np.frexp(np.where(a == 0, 1.0, a) / QMAX[code])
    return np.where(a == 0, 0, np.clip(np.where(m == 0.5, e - 1, e), -127, 127)).astype(np.int64)


def keep(x: np.ndarray, code: str, scale: str):
    """Codes and stored scales of binary32 rows, as bsmm_gated_act keeps them."""
    x = np.asarray(x, np.float32)
    block = 128 if scale == "f32" else 32
    xb = x.reshape(x.shape[0], -1, block)
    absmax = np.abs(xb).max(-1)
    if scale == "ue8m0":
        e = ue8m0_exponent(absmax, code)
        stored, s = (e + 127).astype(np.uint8), np.exp2(e.astype(np.float64)).astype(np.float32)
    else:
        s = absmax * np.float32(1.0 / QMAX[code])  # binary32 product
        s = np.where(absmax == 0, np.float32(1), s) if code == "int8" else np.maximum(s, np.float32(1e-10))
        stored = s
    q = np.clip(div32(xb, s[..., None]), -QMAX[code], QMAX[code]).reshape(x.shape)
    codes = np.rint(q).astype(np.int8) if code == "int8" else F.encode(q, code)
    return codes, stored


def values(codes: np.ndarray, scales: np.ndarray, code: str) -> np.ndarray:
    """binary32(code * scale) of every code."""
    v = codes.astype(np.float64) if code == "int8" else F.decode(codes, code).astype(np.float64)
    s = np.exp2(scales.astype(np.float64) - 127) if scales.dtype == np.uint8 else scales.astype(np.float64)
    v = v.reshape(v.shape[0], s.shape[1], -1) * s[..., None]
    return v.reshape(codes.shape).astype(np.float32)
