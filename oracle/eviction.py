"""Weights that cached keys receive, and the rows kept by them, in float64."""

import numpy as np


def weights(q, lse, k, prev, decay=1.0, window=0, scale=0.0):
    """[Hkv, C]: decay * prev plus the weights from rows q [n, Hq, D] with lse
    [n, Hq] at the last n of the C positions; k [Hkv, C, D], prev [Hkv, C]."""
    n, hq, d = q.shape
    hkv, C, _ = k.shape
    scale = scale if scale > 0 else 1.0 / np.sqrt(d)
    out = np.zeros((hkv, C))
    if prev is not None:
        out[:, :max(0, C - n)] = decay * prev[:, :max(0, C - n)].astype(np.float64)
    for s in range(n):
        at = C - n + s
        lo = 0 if window == 0 else max(0, at - window + 1)
        if at < 0:
            continue
        for h in range(hq):
            if not (np.isfinite(lse[s, h]) and np.isfinite(q[s, h]).all()):
                continue
            g = h // (hq // hkv)
            x = scale * (k[g, lo:at + 1].astype(np.float64) @ q[s, h].astype(np.float64))
            out[g, lo:at + 1] += np.exp(x - np.float64(lse[s, h]))
    return out


def kept(w, keep, sinks, recent):
    """Kept positions of one head with weights w [C], ascending."""
    C = len(w)
    if C <= keep:
        return list(range(C))
    pinned = list(range(sinks)) + list(range(C - recent, C))
    rest = range(sinks, C - recent)
    order = sorted(rest, key=lambda j: (-(w[j] + 0.0) if w[j] == w[j] else np.inf,
                                        w[j] != w[j], j))
    return sorted(pinned + order[:keep - sinks - recent])
