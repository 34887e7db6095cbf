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


def codes(x, s, root=False, step=None):
    """E4M3 codes of x for the scales s; a root that is not zero keeps the
    smallest code.  ``step``: None to round to nearest, or the step whose dither rounds."""
    x = np.asarray(x, np.float32)
    q = div32(x, np.repeat(s, 128)[:x.size])
    if root:
        q = np.where((x > 0) & (q < 2.0 ** -9), np.float32(2.0 ** -9), q)
    if step is not None:
        h = dither(x.size, step)
        q = dithered(q, h >> np.uint32(12) if root else h & np.uint32(0xFFFFF))
    return F.encode(np.clip(q, -448, 448), "e4m3")


def dither(numbers, step):
    """32 bits for each number of a tensor at a step."""
    u = np.uint32
    golden, root3 = u(0x9E3779B9), u(0xBB67AE85)

    def word(x):
        x = (x ^ (x >> u(16))) * golden
        return x ^ (x >> u(15))

    def bits(x, j):
        x = x * root3 + j * golden
        return x ^ (x >> u(16))

    i = np.arange(numbers, dtype=u)
    key = bits(word(np.full(1, step, u)), np.zeros(1, u))
    return bits(word((i >> u(2)) ^ key), i & u(3))


def dithered(q, r):
    """q on E4M3's grid (as if that had no largest number): the number below its
    magnitude, or where the part cut off plus r 2^-20 of a step passes one the number
    above.  A zero has no sign."""
    a = np.abs(np.asarray(q, np.float64))
    step = np.exp2(np.maximum(np.floor(np.log2(np.maximum(a, 2.0 ** -9))), -6) - 3)
    # what the sum of a and 2^-6 keeps in binary32, below 2^-6
    a = np.where(a < 2.0 ** -6, (a.astype(np.float32) + np.float32(2.0 ** -6)).astype(np.float64) - 2.0 ** -6, a)
    low = np.floor(a / step)
    cut = (a / step - low) * 2.0 ** 20
    y = np.copysign((low + (cut + r >= 2.0 ** 20)) * step, q)
    return np.where(y == 0, 0.0, y).astype(np.float32)


def dithers(betas):
    """Whether the library dithers 8-bit states: where a step moves them by less
    than half steps of E4M3."""
    return betas[0] > 17 / 18 or 1 - betas[1] < 2.0 ** -4.5


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
