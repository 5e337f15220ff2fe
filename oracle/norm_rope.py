"""RMS norm of heads, rotation by position, and their gradients, in fp64.

    xhat = x / sqrt(mean(x^2) + eps),  n = xhat w,
    pair (a, b) of n -> (a cos t - b sin t, a sin t + b cos t),  t = position * inv_freq
"""
from __future__ import annotations

import numpy as np


def rotation_pairs(rotary_dim: int, interleaved: bool):
    """Channels (a, b) of every pair."""
    i = np.arange(rotary_dim // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + rotary_dim // 2)


def rotation_angles(positions, inv_freq, sections):
    """positions [axes, B, N] -> angles [B, N, pairs] in fp64."""
    parts, at = [], 0
    for a, n in enumerate(sections):
        parts.append(positions[a].astype(np.float64)[..., None] * inv_freq.astype(np.float64)[at:at + n])
        at += n
    return np.concatenate(parts, -1)


def norm_rope_fp64(x, w, eps, angles=None, interleaved=False):
    """x [B, H, N, d], w [d] or None (no norm), angles [B, N, pairs] or None.
    Returns (y, magnitude): |a| + |b| of every value's pair (|n| where not
    rotated), the size that the rounding errors of the rotation go by."""
    n = x.astype(np.float64)
    if w is not None:
        n = n / np.sqrt(np.mean(n * n, -1, keepdims=True) + eps) * w.astype(np.float64)
    y, mag = n.copy(), np.abs(n)
    if angles is not None and angles.shape[-1]:
        ia, ib = rotation_pairs(2 * angles.shape[-1], interleaved)
        c, s = np.cos(angles)[:, None], np.sin(angles)[:, None]
        y[..., ia] = n[..., ia] * c - n[..., ib] * s
        y[..., ib] = n[..., ia] * s + n[..., ib] * c
        mag[..., ia] = mag[..., ib] = np.abs(n[..., ia]) + np.abs(n[..., ib])
    return y, mag


def norm_rope_bwd_fp64(x, w, eps, dy, angles=None, interleaved=False):
    """Gradients (dx, dw or None) of sum(y * dy) for norm_rope_fp64's y."""
    g = dy.astype(np.float64).copy()
    if angles is not None and angles.shape[-1]:
        ia, ib = rotation_pairs(2 * angles.shape[-1], interleaved)
        c, s = np.cos(angles)[:, None], np.sin(angles)[:, None]
        ga, gb = g[..., ia].copy(), g[..., ib].copy()
        g[..., ia] = ga * c + gb * s
        g[..., ib] = gb * c - ga * s
    if w is None:
        return g, None
    x = x.astype(np.float64)
    r = 1.0 / np.sqrt(np.mean(x * x, -1, keepdims=True) + eps)
    xhat = x * r
    dw = (g * xhat).sum((0, 1, 2))
    g = g * w.astype(np.float64)
    return r * (g - xhat * np.mean(g * xhat, -1, keepdims=True)), dw
