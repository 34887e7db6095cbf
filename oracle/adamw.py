"""AdamW, float64, and its 8-bit states (oracle; test infrastructure)."""

from __future__ import annotations

import numpy as np

from . import formats as F
from .quantize import div32


def step(p, g, m, v, t, lr, betas, eps, weight_decay, grad_scale=1.0):
    """(p, m, v) after step t, from the textbook form."""
    p, g, m, v = (np.asarray(x, np.float64) for x in (p, g, m, v))
    g = grad_scale * g
    m = betas[0] * m + (1 - betas[0]) * g
    v = betas[1] * v + (1 - betas[1]) * g * g
    hat_m, hat_v = m / (1 - betas[0] ** t), v / (1 - betas[1] ** t)
    return p - lr * (hat_m / (np.sqrt(hat_v) + eps) + weight_decay * p), m, v


def scales(x):
    """Binary32 scale of each 128 numbers (the last block may be shorter)."""
    x = np.asarray(x, np.float32)
    top = np.abs(np.concatenate([x, np.zeros(-x.size % 128, np.float32)])).reshape(-1, 128).max(1)
    s = np.maximum(top * np.float32(1.0 / 448.0), np.float32(2.0 ** -126))
    return np.where(top == 0, np.float32(1), s).astype(np.float32)


def codes(x, s, root=False):
    """E4M3 codes of x for the scales s; a root that is not zero keeps the smallest code."""
    x = np.asarray(x, np.float32)
    q = np.clip(div32(x, np.repeat(s, 128)[:x.size]), -448, 448)
    c = F.encode(q, "e4m3")
    return np.where((x > 0) & (c == 0), 1, c).astype(np.uint8) if root else c


def values(c, s):
    """binary32(code * scale)."""
    return (F.decode(c, "e4m3").astype(np.float32) * np.repeat(s, 128)[:c.size]).astype(np.float32)


def step32(p, g, m, v, t, lr, betas, eps, weight_decay, grad_scale=1.0):
    """(p, m, v) with every operation rounded to binary32 on its own, as the
    library's entry point defines them."""
    f = np.float32
    p, g, m, v = (np.asarray(x, f) for x in (p, g, m, v))
    decay, rate = f(1.0 - lr * weight_decay), f(lr / (1.0 - betas[0] ** t))
    root2 = f(1.0 / np.sqrt(1.0 - betas[1] ** t))
    g = g * f(grad_scale)
    m = f(betas[0]) * m + f(1.0 - betas[0]) * g
    v = f(betas[1]) * v + (f(1.0 - betas[1]) * g) * g
    d = np.sqrt(v) * root2 + f(eps)
    return p * decay - rate * (m / d), m, v
