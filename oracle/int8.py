"""The 8-bit cache with one scale per block of 64 positions and head, oracle
side (test infrastructure only).

A library addition without a counterpart in the pages: beside the Q4_0 and
F16 caches, K and V held as signed 8-bit codes. The definition, in float64:

* rows are bf16 values; a block of 64 positions of one head is quantised when
  it is complete: ``amax = max |x|``, ``code = round-half-even(127 x / amax)``,
  ``value = code * amax / 127``; a block with ``amax < 2^-40`` is all zeros;
* the open block's rows are their bf16 values.

So the cache's values are a function of the committed rows alone, however
they arrived.
"""

import numpy as np

BLOCK = 64
SMALL = 2.0 ** -40


def encode_blocks(rows):
    """Codes (int8 [Hkv, nb, 64, D]) and float32 scales [Hkv, nb] of the
    complete blocks of ``rows`` [Hkv, n, D] (bf16 values)."""
    rows = np.asarray(rows, dtype=np.float64)
    hkv, n, d = rows.shape
    nb = n // BLOCK
    x = rows[:, :nb * BLOCK].reshape(hkv, nb, BLOCK, d)
    amax = np.abs(x).max(axis=(2, 3)) if nb else np.zeros((hkv, 0))
    codes = np.zeros(x.shape, np.int8)
    for h in range(hkv):
        for b in range(nb):
            if amax[h, b] >= SMALL:
                codes[h, b] = np.rint(127.0 * x[h, b] / amax[h, b]).astype(np.int8)
    scale = np.where(amax >= SMALL, amax.astype(np.float32) / np.float32(127.0),
                     np.float32(0.0)).astype(np.float32)
    return codes, scale


def cached_values(rows):
    """float64 values [Hkv, n, D] of a cache with ``rows`` committed: code *
    scale (the float32 scale that is stored) and the open block's rows."""
    rows = np.asarray(rows, dtype=np.float64)
    codes, scale = encode_blocks(rows)
    out = rows.copy()
    nb = codes.shape[1]
    v = codes.astype(np.float64) * scale.astype(np.float64)[:, :, None, None]
    out[:, :nb * BLOCK] = v.reshape(rows.shape[0], nb * BLOCK, rows.shape[2])
    return out


def unpack_k(codes):
    """[Hkv, nb, D/16, 64, 16] (K layout) as [Hkv, nb, 64, D]."""
    h, nb, p, t, e = codes.shape
    return codes.transpose(0, 1, 3, 2, 4).reshape(h, nb, t, p * e)


def unpack_v(codes):
    """[Hkv, nb, 4, D, 16] (V layout) as [Hkv, nb, 64, D]."""
    h, nb, g, d, e = codes.shape
    return codes.transpose(0, 1, 2, 4, 3).reshape(h, nb, g * e, d)
