"""Norm and rotation of queries and keys, from the definition in float64."""

import numpy as np


def depths(parent):
    """Depth of each node; an entry outside [0, i) counts as 0."""
    d = [0] * len(parent)
    for i in range(1, len(parent)):
        p = int(parent[i])
        d[i] = d[p if 0 <= p < i else 0] + 1
    return np.array(d, dtype=np.int64)


def norm(x, weight, eps):
    x = np.asarray(x, dtype=np.float64)
    with np.errstate(all="ignore"):
        y = x / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps)
    return y if weight is None else y * np.asarray(weight, dtype=np.float64)


def rotate(y, positions, inv_freq, interleaved):
    """y [N, H, D]; pair i turned by positions[n] * inv_freq[i] rad."""
    half = len(inv_freq)
    out = np.array(y, dtype=np.float64)
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        t = np.asarray(positions, dtype=np.float64) * float(inv_freq[i])
        c, s = np.cos(t)[:, None], np.sin(t)[:, None]
        out[..., a] = y[..., a] * c - y[..., b] * s
        out[..., b] = y[..., b] * c + y[..., a] * s
    return out
