"""Rotary positions in float64, pair by pair as complex numbers.  TEST INFRASTRUCTURE ONLY."""
import numpy as np


def rope(x, positions, inv_freq, interleaved=False, factor=1.0, inverse=False):
    """x [T, H, D] with the first 2 len(inv_freq) values of each head turned by +-positions *
    inv_freq and scaled by factor; the rest copied."""
    x = np.asarray(x, dtype=np.float64)
    f = np.asarray(inv_freq, dtype=np.float64)
    n = len(f)
    angle = np.asarray(positions, dtype=np.float64)[:, None] * f[None]
    z = factor * np.exp((-1j if inverse else 1j) * angle)[:, None, :]
    y = x.copy()
    re = np.arange(n) * 2 if interleaved else np.arange(n)
    im = re + 1 if interleaved else re + n
    w = (x[..., re] + 1j * x[..., im]) * z
    y[..., re], y[..., im] = w.real, w.imag
    return y


def freqs(rot_dim, theta, scaling="none", factor=1.0, orig_len=0, beta_fast=32.0, beta_slow=1.0):
    """(inverse frequencies, attention factor); "ramp" mixes by the pair's index."""
    f = np.array([theta ** (-2.0 * i / rot_dim) for i in range(rot_dim // 2)])
    if scaling == "none":
        return f, 1.0
    if scaling == "linear":
        return f / factor, 1.0
    # pair i turns orig_len f_i / 2 pi times; the border indices are rounded outwards
    index = lambda turns: rot_dim * np.log(orig_len / (2 * np.pi * turns)) / (2 * np.log(theta))  # noqa: E731
    lo, hi = max(np.floor(index(beta_fast)), 0), min(np.ceil(index(beta_slow)), rot_dim - 1)
    out = []
    for i in range(rot_dim // 2):
        r = min(max((i - lo) / max(hi - lo, 1e-3), 0.0), 1.0)
        out.append(f[i] * (1 - r) + f[i] / factor * r)
    return np.array(out), 0.1 * np.log(factor) + 1.0
