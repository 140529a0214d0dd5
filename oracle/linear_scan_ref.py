"""fp64 reference of the gated linear recurrence, test infrastructure only.

Per channel, step by step: h_t = a_t h_{t-1} + b_t x_t, y_t = h_t.  Packed
sequences are a loop over their ranges.  The gradient is the adjoint recursion
of the same loop.  All arithmetic is fp64 NumPy.
"""
from __future__ import annotations

import numpy as np


def forward(a, x, b=None, h0=None):
    """a, x, b [T, D]; h0 [D].  Returns (y [T, D], h_T [D])."""
    T, D = a.shape
    h = np.zeros(D) if h0 is None else np.array(h0, np.float64)
    y = np.empty((T, D))
    for t in range(T):
        h = a[t] * h + (x[t] if b is None else b[t] * x[t])
        y[t] = h
    return y, h


def backward(a, x, y, dy, b=None, h0=None, dh_T=None):
    """Gradients (a, x, b or None, h0) given y (as stored) and dy, dh_T."""
    T, D = a.shape
    c = np.zeros(D) if dh_T is None else np.array(dh_T, np.float64)
    da, dx = np.empty((T, D)), np.empty((T, D))
    db = None if b is None else np.empty((T, D))
    for t in range(T - 1, -1, -1):
        g = dy[t] + c
        before = y[t - 1] if t > 0 else (np.zeros(D) if h0 is None else h0)
        da[t] = g * before
        dx[t] = g if b is None else g * b[t]
        if b is not None:
            db[t] = g * x[t]
        c = a[t] * g
    return da, dx, db, c


def forward_bound(a, x, b=None, h0=None):
    """Per element, the sum of what |rounding| each operation may add, in units
    of one relative rounding: the recurrence on absolute values, where every
    step adds a rounding of the product of gates and one of the sum to all
    earlier contributions, and a new contribution starts with a few (its own
    product, and the sums where tiles meet)."""
    T, D = a.shape
    m = np.zeros(D) if h0 is None else np.abs(h0)   # magnitudes
    e = 8 * m
    out = np.empty((T, D))
    for t in range(T):
        u = np.abs(x[t] if b is None else b[t] * x[t])
        e = np.abs(a[t]) * (e + 2 * m) + 8 * u
        m = np.abs(a[t]) * m + u
        out[t] = e
    return out, e


def backward_bound(a, dy, dh_T=None):
    """The same for g (per step) and c (at the end)."""
    T, D = a.shape
    m = np.zeros(D) if dh_T is None else np.abs(dh_T)
    e = 8 * m
    out = np.empty((T, D))
    for t in range(T - 1, -1, -1):
        m = m + np.abs(dy[t])
        e = e + 8 * np.abs(dy[t])
        out[t] = e
        e = np.abs(a[t]) * (e + 2 * m)
        m = np.abs(a[t]) * m
    return out, e
