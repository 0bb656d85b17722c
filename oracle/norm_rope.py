"""Norms of heads with the rotary positions behind them, float64, and the gradient.  TEST INFRASTRUCTURE ONLY."""
import numpy as np

from .rope import rope


def norm(x, weight, eps, offset=0.0):
    x = np.asarray(x, dtype=np.float64)
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    return x * r * (1.0 if weight is None else weight + offset)


def norm_rope(x, weight, eps, pos, inv_freq, interleaved=False, factor=1.0, offset=0.0):
    y = norm(x, weight, eps, offset)
    return y if inv_freq is None else rope(y, pos, inv_freq, interleaved, factor)


def norm_rope_grad(dy, x, weight, eps, pos, inv_freq, interleaved=False, factor=1.0, offset=0.0):
    """(dx, dw, sizes of dx's parts, of dw's terms)."""
    dy, x = np.asarray(dy, dtype=np.float64), np.asarray(x, dtype=np.float64)
    g = dy if inv_freq is None else rope(dy, pos, inv_freq, interleaved, factor, True)
    w = 1.0 if weight is None else weight + offset
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    u = g * w
    dx = r * (u - x * r * r * (u * x).mean(-1, keepdims=True))
    size = r * (np.abs(u) + np.abs(x) * r * r * np.abs(u * x).mean(-1, keepdims=True))
    return dx, (g * x * r).sum((0, 1)), size, np.abs(g * x * r).sum((0, 1))
