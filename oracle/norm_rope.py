"""Root-mean-square norm per head and the rotation of its pairs by position, and the gradients, from the definition.

``x`` is [batch, len, heads, dim], ``pos`` [batch, len] integers, ``freqs`` radians per position of each pair.
"""

from __future__ import annotations

import numpy as np


def pairs(dim, n, interleaved):
    """Index arrays (first, second) of the n rotated pairs."""
    i = np.arange(n)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + n)


def rotate(x, pos, freqs, interleaved, sign=1.0):
    """The rotation as a complex product: (a + i b) e^(i sign pos freq)."""
    a, b = pairs(x.shape[-1], len(freqs), interleaved)
    z = np.exp(1j * sign * pos.astype(np.float64)[..., None] * np.asarray(freqs))[:, :, None, :]
    turned = (x[..., a] + 1j * x[..., b]) * z
    y = np.array(x, dtype=np.float64)
    y[..., a], y[..., b] = turned.real, turned.imag
    return y


def forward(x, weight, pos, freqs, eps, interleaved):
    n = x / np.sqrt((x * x).mean(axis=-1, keepdims=True) + eps) * weight
    return rotate(n, pos, freqs, interleaved)


def backward(x, weight, pos, freqs, eps, interleaved, dy):
    """(dx, dweight)."""
    rstd = 1.0 / np.sqrt((x * x).mean(axis=-1, keepdims=True) + eps)
    hat = x * rstd
    g = rotate(dy, pos, freqs, interleaved, -1.0)
    h = g * weight
    return rstd * (h - hat * (h * hat).mean(axis=-1, keepdims=True)), (g * hat).sum(axis=(0, 1, 2))


def error_bounds(x, weight, pos, freqs, eps, interleaved, dy, u_out, abs_out=0.0):
    """Largest elementwise errors of (y, dx, dweight) of a float32 evaluation with results rounded to relative u_out,
    or to absolute abs_out below the type's normal range.

    cos and sin are off by at most 4e-7 (the angle's rounding to 2^-25 turns, the functions' 1.3e-7); the norm's sum
    over the head by D 2^-24, each further operation by 2^-24 of its operands.
    """
    f, D = 2.0 ** -24, x.shape[-1]
    e = (D + 16) * f + 4e-7
    rstd = 1.0 / np.sqrt((x * x).mean(axis=-1, keepdims=True) + eps)
    hat = x * rstd
    a, b = pairs(D, len(freqs), interleaved)

    def both(t):  # |a| + |b| of the pair
        r = np.abs(t)
        s = r.copy()
        s[..., a], s[..., b] = r[..., a] + r[..., b], r[..., a] + r[..., b]
        return s

    y = forward(x, weight, pos, freqs, eps, interleaved)
    t_y = abs_out + u_out * np.abs(y) + e * both(hat * weight)
    dx, _ = backward(x, weight, pos, freqs, eps, interleaved, dy)
    g = both(dy)
    t_dx = abs_out + u_out * np.abs(dx) + 4 * e * rstd * (g * np.abs(weight) + np.abs(hat) * (g * np.abs(weight * hat)).mean(
        axis=-1, keepdims=True))
    rows = x[..., 0].size
    t_dw = ((2 * e + (rows + 64) * f) * g * np.abs(hat)).sum(axis=(0, 1, 2))
    return t_y, t_dx, t_dw
