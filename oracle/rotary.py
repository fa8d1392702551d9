"""Rotary positions in numpy (include/asffn.h), angles in extended precision."""
from __future__ import annotations

import numpy as np


def frequencies(rot_dim: int, base: float, scaling: str = "none", factor: float = 1.0, original: float = 4096.0):
    """(radians per position of each pair, scale), from the formulas."""
    i = np.arange(rot_dim // 2, dtype=np.float64)
    if scaling == "ntk" and rot_dim > 2:
        base = base * factor ** (rot_dim / (rot_dim - 2))
    f = base ** (-2 * i / rot_dim)
    if scaling == "linear":
        return f / factor, 1.0
    if scaling == "yarn":
        pair = lambda turns: rot_dim * np.log(original / (2 * np.pi * turns)) / (2 * np.log(base))  # noqa: E731
        low, high = max(np.floor(pair(32.0)), 0.0), min(np.ceil(pair(1.0)), rot_dim - 1.0)
        m = np.clip((i - low) / max(high - low, 0.001), 0, 1)
        return (1 - m) * f + m * f / factor, 1 + 0.1 * np.log(factor)
    return f, 1.0


def turn(x, pos, freq, scale: float, layout: str):
    """(y, |u| + |w| of each turned element's pair) for x [T, heads, D]; columns behind the pairs pass."""
    n = len(freq)
    a = np.asarray(pos, np.longdouble)[:, None] * np.asarray(freq, np.longdouble)
    a = a - np.round(a / (2 * np.longdouble("3.14159265358979323846264338327950288"))) \
        * (2 * np.longdouble("3.14159265358979323846264338327950288"))
    cos, sin = (f(a).astype(np.float64)[:, None] * scale for f in (np.cos, np.sin))
    x = np.asarray(x, np.float64)
    at, to = (slice(0, n), slice(n, 2 * n)) if layout == "half" else (slice(0, 2 * n, 2), slice(1, 2 * n, 2))
    y, size = x.copy(), np.zeros_like(x)
    u, w = x[..., at], x[..., to]
    y[..., at], y[..., to] = u * cos - w * sin, w * cos + u * sin
    size[..., at] = size[..., to] = np.abs(u) + np.abs(w)
    return y, size
