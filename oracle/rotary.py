"""Rotary positions (oracle side; test infrastructure only): float64, pair by pair."""

from __future__ import annotations

import numpy as np


def rotate(x, positions, inv_freq, axes=None, interleaved=False, scale=1.0):
    """Rows x [T, heads, dim] turned by positions [T] or [axes, T]: (float64 rows, magnitudes).

    ``magnitudes`` is |x1 c| + |x2 s| of each element (0 where nothing turns): what rounding bounds scale with.
    """
    x = np.asarray(x, np.float64)
    positions = np.atleast_2d(np.asarray(positions, np.float64))
    n = len(inv_freq)
    out, mag = x.copy(), np.zeros_like(x)
    for i in range(n):
        a = positions[0 if axes is None else int(axes[i])] * float(inv_freq[i])
        c, s = scale * np.cos(a)[:, None], scale * np.sin(a)[:, None]
        p, q = (2 * i, 2 * i + 1) if interleaved else (i, n + i)
        x1, x2 = x[..., p], x[..., q]
        out[..., p], out[..., q] = x1 * c - x2 * s, x2 * c + x1 * s
        mag[..., p], mag[..., q] = np.abs(x1 * c) + np.abs(x2 * s), np.abs(x2 * c) + np.abs(x1 * s)
    return out, mag
