"""Oracle: rotary positions (test infrastructure), plain NumPy in 64 bits.

Pair (x, y) of a head's first R values at position p becomes scale * (x cos w - y sin w, y cos w + x sin w), w = p *
inv_freq[j]; pair j is (x[j], x[j + R / 2]), or (x[2 j], x[2 j + 1]) interleaved.  A chain's node v stands at position
len + v, a tree's at len plus the number of its ancestors (a parent outside [0, v) makes a root).

Parity unpinned by the pages: they name no positions.
"""
from __future__ import annotations

import numpy as np


def depths(parent):
    out = []
    for v, p in enumerate(parent):
        out.append(out[p] + 1 if 0 <= p < v else 0)
    return np.array(out, dtype=np.int64)


def rotate(x, position, inv_freq, scale=1.0, interleaved=False):
    """x [n, H, D] (float64) at position [n] -> (the rotated rows, the size of what each value adds up)."""
    half = len(inv_freq)
    w = position.astype(np.float64)[:, None, None] * inv_freq
    c, s = scale * np.cos(w), scale * np.sin(w)
    a = np.arange(half) * (2 if interleaved else 1)
    b = a + (1 if interleaved else half)
    out, size = x.astype(np.float64).copy(), np.abs(x.astype(np.float64))
    out[..., a], out[..., b] = x[..., a] * c - x[..., b] * s, x[..., b] * c + x[..., a] * s
    both = abs(scale) * (np.abs(x[..., a]) + np.abs(x[..., b]))
    size[..., a] = size[..., b] = both
    return out, size
