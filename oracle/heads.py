"""Norms and position rotation of query and key heads in float64 (oracle; test infrastructure
only): per head RMS norm or layer norm, then the rotation of `rot` values from rot_begin on, pairs
half the rotated width apart or neighbours.

Every function also returns the scale of a value's rounding error in fp32: the magnitudes that went
into it.

Pinned by: hand-worked heads, and the rotation's invariants (lengths of pairs kept, angles add).
"""

import numpy as np


def norm(x, kind, weight=None, bias=None, eps=1e-6):
    """x [..., D]; kind "none", "rms" or "layer".  (values, error scale)"""
    x = np.asarray(x, np.float64)
    d = x.shape[-1]
    w = np.ones(d) if weight is None else np.asarray(weight, np.float64)
    b = np.zeros(d) if bias is None else np.asarray(bias, np.float64)
    if kind == "none":
        return x, np.abs(x)
    spread = np.zeros(x.shape[:-1] + (1,))
    y = x
    if kind == "layer":
        y = x - x.mean(-1, keepdims=True)
        spread = np.abs(x).mean(-1, keepdims=True)
    r = 1.0 / np.sqrt((y * y).mean(-1, keepdims=True) + eps)
    return y * r * w + b, np.abs(w) * r * (np.abs(x) + spread) * (1 + spread * r) + np.abs(b)


def rotate(x, scale, pos, cos_sin, rot_begin=0, interleaved=False):
    """x [tokens, heads, D] turned by row pos[t] of cos_sin [positions, rot]."""
    x, scale = x.copy(), scale.copy()
    rot = cos_sin.shape[1]
    half = rot // 2
    i = np.arange(half)
    u, v = (rot_begin + 2 * i, rot_begin + 2 * i + 1) if interleaved else (rot_begin + i, rot_begin + half + i)
    c = np.asarray(cos_sin[pos, :half], np.float64)[:, None, :]
    s = np.asarray(cos_sin[pos, half:], np.float64)[:, None, :]
    a, b, p, q = x[..., u], x[..., v], scale[..., u], scale[..., v]
    x[..., u], x[..., v] = a * c - b * s, b * c + a * s
    scale[..., u], scale[..., v] = p * np.abs(c) + q * np.abs(s), q * np.abs(c) + p * np.abs(s)
    return x, scale
