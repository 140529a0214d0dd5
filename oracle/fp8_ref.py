"""fp64 reference of the e4m3 block format and its product, test
infrastructure only.  A block's scale is max(largest magnitude, 2^-100) / 448;
a code is the nearest e4m3 number to value / scale, ties to the even one.
"""
from __future__ import annotations

import numpy as np

FLOOR = 2.0 ** -100


def e4m3(v):
    """The nearest e4m3 number: 3 fraction bits, exponents from 2^-6 (below it
    steps of 2^-9), largest 448."""
    v = np.clip(np.asarray(v, np.float64), -448.0, 448.0)
    _, e = np.frexp(v)
    unit = np.ldexp(1.0, np.maximum(e - 1, -6) - 3)
    return np.round(v / unit) * unit


def scales(x, tile=False):
    """Scales of a matrix's blocks of 128 along its rows, or of its tiles."""
    rows, cols = x.shape
    kb, rb = -(-cols // 128), -(-rows // 128)
    top = np.zeros((rb if tile else rows, kb))
    for k in range(kb):
        part = np.abs(x[:, 128 * k:128 * (k + 1)])
        if tile:
            for r in range(rb):
                top[r, k] = part[128 * r:128 * (r + 1)].max()
        else:
            top[:, k] = part.max(1)
    return np.maximum(top, FLOOR) / 448.0


def spread(s, rows, cols, tile=False):
    """One scale per element."""
    s = np.repeat(s, 128, 1)[:, :cols]
    return np.repeat(s, 128, 0)[:rows] if tile else s


def matmul(x, sx, w, sw, tile):
    """(out, sum of absolute values) of the scaled product x w^T."""
    xs = x * spread(sx, *x.shape)
    ws = w * spread(sw, *w.shape, tile)
    return xs @ ws.T, np.abs(xs) @ np.abs(ws).T
