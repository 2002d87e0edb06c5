"""Norm of each head with rotary positions and its gradients, in plain fp64 NumPy
from the definitions (test infrastructure only).

Forward: R(x r w), r = 1 / sqrt(mean(x^2) + eps), R the rotation of oracle.cache.
Gradients, with g the output's gradient times R transposed:
dw = sum g x r, dx = r (g w - x r mean(g w x r)).
"""
from __future__ import annotations

import numpy as np

from .cache import rope


def _unit(x, eps):
    r = 1.0 / np.sqrt(np.mean(x * x, -1, keepdims=True) + eps)
    return x * r, r


def forward(x, w, positions, freqs, interleaved=False, mscale=1.0, eps=1e-6):
    """x [B, H, N, d], w [d] or None."""
    u, _ = _unit(np.asarray(x, np.float64), eps)
    return rope(u if w is None else u * w, positions, freqs, interleaved, mscale)


def backward(dy, x, w, positions, freqs, interleaved=False, mscale=1.0, eps=1e-6):
    """(dx [B, H, N, d], dw [d])."""
    u, r = _unit(np.asarray(x, np.float64), eps)
    g = rope(dy, positions, freqs, interleaved, mscale, inverse=True)
    dw = (g * u).sum((0, 1, 2))
    if w is not None:
        g = g * w
    return r * (g - u * np.mean(g * u, -1, keepdims=True)), dw


def pair_magnitudes(x, freqs_n, interleaved):
    """|x|, and for the elements of a pair |x| + |y|: what a rotation's rounding errors
    are relative to."""
    mag = np.abs(np.asarray(x, np.float64))
    out = mag.copy()
    n = freqs_n
    first = 2 * np.arange(n) if interleaved else np.arange(n)
    second = first + 1 if interleaved else first + n
    out[..., first] = out[..., second] = mag[..., first] + mag[..., second]
    return out
