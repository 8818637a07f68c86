"""Per-head RMS norm with rotation and its gradients in float64 (numpy), from the
definition: each pair as one complex number."""
from __future__ import annotations

import numpy as np


def _angles(pos, freq):
    return pos[:, None, :, None].astype(np.float64) * freq  # [B, 1, N, rot / 2]


def _pairs(rot, interleaved):
    i = np.arange(rot // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, rot // 2 + i)


def _turn(y, pos, freq, interleaved, sign=1.0):
    a, b = _pairs(2 * len(freq), interleaved)
    z = (y[..., a] + 1j * y[..., b]) * np.exp(1j * sign * _angles(pos, freq))
    out = y.copy()
    out[..., a], out[..., b] = z.real, z.imag
    return out


def norm_rope(x, w, pos, freq, eps, interleaved):
    """x [B, H, N, D], w [D], pos [B, N], freq [rot / 2] radians a position."""
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    return _turn(x * r * w, pos, freq, interleaved)


def norm_rope_bwd(x, w, dy, pos, freq, eps, interleaved):
    """dx, dw, and the magnitude sum of dw's terms."""
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    n = x * r
    g = _turn(dy, pos, freq, interleaved, -1.0)
    gw = g * w
    dx = r * (gw - n * (gw * n).mean(-1, keepdims=True))
    return dx, (g * n).sum((0, 1, 2)), np.abs(g * n).sum((0, 1, 2))
